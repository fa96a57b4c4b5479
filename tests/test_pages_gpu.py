"""The operators on the pages of a cache, against the same operators written out in Python:
equal tables, lengths and references, and equal bits in both pools."""
import random

import pytest
import torch

from gqa_attention_forward_gb300 import binding
from packed_util import DT, offsets
from paged_util import Model, build

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def status():
    return binding.attn_last_device_error(torch.cuda.current_stream())


@pytest.mark.parametrize("page,Hkv,D,layers,dtype", [(16, 1, 64, 1, "f16"), (32, 3, 128, 2, "bf16"),
                                                     (128, 8, 128, 1, "bf16"), (256, 2, 64, 3, "f16")])
def test_fork_free_copy_compact(page, Hkv, D, layers, dtype):
    lens = [5 * page + 3, page, 1, 2 * page - 1, 0, 3 * page, 7]
    c = build(lens, page, Hkv, D, dtype, layers, extra_pages=12, seed=page, n_rows=20)
    m = Model(c)
    pa, ch = [0, 0, 2, 5, 4, 3, 0], [10, 7, 8, 9, 12, 19, 11]  # a parent many times, an empty parent
    binding.kv_fork(c, i32(pa), i32(ch))
    m.fork(pa, ch)
    m.same(c)
    gone = [0, 8, 3, 3, 12, 15]  # one twice, empty ones
    binding.kv_free(c, i32(gone))
    m.free(dict.fromkeys(gone))
    m.same(c)
    free = [p for p, r in enumerate(m.refs) if r == 0][:3]
    src = [p for p, r in enumerate(m.refs) if r > 0][:len(free)]
    binding.kv_copy(c, i32(src), i32(free))
    m.copy(src, free)
    m.same(c)
    live = binding.kv_compact(c)
    assert int(live) == m.compact()
    m.same(c)
    m.consistent()
    assert int(binding.kv_compact(c)) == int(live)  # already dense
    m.same(c)
    assert status() == binding.ATTN_OK


@pytest.mark.parametrize("page", [16, 64])
def test_extend_append_accept(page):
    """Growing sequences a step at a time: none, one, several pages; rows cut from a projection."""
    Hkv, D, layers = 2, 128, 2
    c = binding.KVPages.empty(layers, 40, Hkv, page, D, 6, 12, torch.bfloat16)
    c.k.fill_(1.0)
    c.v.fill_(2.0)
    m = Model(c)
    rng = random.Random(page)
    for step in range(8):
        seqs = rng.sample(range(6), rng.randint(1, 6)) if step % 2 else None
        ids = list(range(6)) if seqs is None else seqs
        new = [rng.choice([0, 1, 1, 5, 8, page]) for _ in ids]
        binding.kv_extend(c, i32(new), None if seqs is None else i32(seqs))
        m.extend(ids, new)
        x = torch.randn(sum(new) + 2, 2 * Hkv + 1, D, device="cuda").to(torch.bfloat16)  # two rows too many
        for layer in range(layers):
            k_new, v_new = x[:, :Hkv], x[:, Hkv + 1:]
            binding.kv_append(c, k_new, v_new, offsets(new), None if seqs is None else i32(seqs), layer=layer)
            m.append(layer, ids, k_new, v_new, new)
        m.same(c)
        paths = [sorted(rng.sample(range(t), rng.randint(0, t))) for t in new]
        width = max(1, max(len(p) for p in paths) + step % 2)
        binding.kv_accept(c, offsets(new), i32([p + [-1] * (width - len(p)) for p in paths]).view(len(ids), width),
                          i32([len(p) for p in paths]), None if seqs is None else i32(seqs))
        m.accept(ids, new, paths)
        m.same(c)
    m.consistent()
    assert status() == binding.ATTN_OK


def test_accept_of_the_largest_tree():
    c = build([128 + 77, 128], 32, 3, 64, "f16", 5, seed=2)
    m = Model(c)
    paths = [list(range(1, 128)), [0, 1, 2, 64, 127]]
    binding.kv_accept(c, offsets([128, 128]), i32([p + [0] * (127 - len(p)) for p in paths]), i32([127, 5]))
    m.accept([0, 1], [128, 128], paths)
    m.same(c)


def test_pool_runs_out():
    """Requests are served in order until the free pages do not hold one; from there on nothing
    changes and the error word says so."""
    page = 16
    c = build([page, 3, 20], page, 1, 64, "f16", extra_pages=2, width=8, n_rows=8)
    m = Model(c)
    binding.kv_extend(c, i32([page, 2 * page, 1]), i32([0, 1, 2]))  # one page, then two of the one left
    m.extend([0, 1, 2], [page, 2 * page, 1])
    m.same(c)
    assert m.lens[0] == 2 * page and m.lens[1] == 3 and m.lens[2] == 20
    assert status() == binding.ATTN_ERR_POOL
    binding.kv_fork(c, i32([1, 2, 0]), i32([3, 4, 5]))  # the second has no page left
    m.fork([1, 2, 0], [3, 4, 5])
    m.same(c)
    assert m.lens[3] == 3 and m.lens[4] == 0 and m.lens[5] == 0
    assert status() == binding.ATTN_ERR_POOL
    binding.kv_free(c, i32([1, 3]))
    m.free([1, 3])
    m.same(c)
    assert status() == binding.ATTN_OK


def test_large_pool_and_many_sequences():
    """More pages than one pass of the page search takes, more sequences than a block has
    threads, and most pages used."""
    page, n = 16, 1500
    lens = [1 + (37 * i) % 70 for i in range(n)]
    c = build(lens, page, 1, 64, "bf16", extra_pages=900, seed=4, n_rows=2 * n)
    m = Model(c)
    gone = list(range(0, n, 3))
    binding.kv_free(c, i32(gone))
    m.free(gone)
    pa, ch = list(range(1, n, 3)), [n + i for i in range(len(range(1, n, 3)))]
    binding.kv_fork(c, i32(pa), i32(ch))
    m.fork(pa, ch)
    m.same(c)
    new = [(11 * i) % 40 for i in range(n)]
    assert status() == binding.ATTN_OK
    binding.kv_extend(c, i32(new))
    fits = m.extend(range(n), new)  # they do not: the last requests are not served
    m.same(c)
    assert not fits and status() == binding.ATTN_ERR_POOL
    live = binding.kv_compact(c)
    # as Model.compact, with one renaming of the table
    total = sum(r > 0 for r in m.refs)
    holes = [p for p in range(total) if m.refs[p] == 0]
    movers = [p for p in range(total, len(m.refs)) if m.refs[p] > 0]
    m.copy(movers, holes)
    to = dict(zip(movers, holes))
    for a, b in to.items():
        m.refs[b], m.refs[a] = m.refs[a], 0
    m.table = [[to.get(x, x) for x in r] for r in m.table]
    assert int(live) == total
    m.same(c)
    m.consistent()
    assert status() == binding.ATTN_OK


BAD = [
    ("extend", binding.ATTN_ERR_SHAPE, lambda c: binding.kv_extend(c, i32([1, 1]), i32([0, 99]))),
    ("extend", binding.ATTN_ERR_SHAPE, lambda c: binding.kv_extend(c, i32([-1]), i32([0]))),
    ("extend", binding.ATTN_ERR_SHAPE, lambda c: binding.kv_extend(c, i32([10 ** 6]), i32([0]))),
    ("fork", binding.ATTN_ERR_SHAPE, lambda c: binding.kv_fork(c, i32([0]), i32([1]))),  # not empty
    ("fork", binding.ATTN_ERR_SHAPE, lambda c: binding.kv_fork(c, i32([-1]), i32([4]))),
    ("fork", binding.ATTN_ERR_SHAPE, lambda c: binding.kv_fork(c, i32([4]), i32([4]))),
    ("free", binding.ATTN_ERR_SHAPE, lambda c: binding.kv_free(c, i32([77]))),
    ("copy", binding.ATTN_ERR_PAGE, lambda c: binding.kv_copy(c, i32([0]), i32([10 ** 6]))),
    ("copy", binding.ATTN_ERR_PAGE, lambda c: binding.kv_copy(c, i32([-2]), i32([0]))),
    ("append", binding.ATTN_ERR_SHAPE, lambda c: binding.kv_append(c, *new(c, 500), i32([0, 500]), i32([0]))),
    ("append", binding.ATTN_ERR_SHAPE, lambda c: binding.kv_append(c, *new(c, 2), i32([0, 2]), i32([-1]))),
    ("append", binding.ATTN_ERR_SHAPE, lambda c: binding.kv_append(c, *new(c, 2), i32([0, 5]), i32([0]))),
    ("append", binding.ATTN_ERR_SHAPE, lambda c: binding.kv_append(c, *new(c, 2), i32([-3, 2]), i32([0]))),
    ("accept", binding.ATTN_ERR_SHAPE, lambda c: binding.kv_accept(c, i32([0, 4]), i32([[1, 1]]), i32([2]))),
    ("accept", binding.ATTN_ERR_SHAPE, lambda c: binding.kv_accept(c, i32([0, 4]), i32([[1, 4]]), i32([2]))),
    ("accept", binding.ATTN_ERR_SHAPE, lambda c: binding.kv_accept(c, i32([0, 4]), i32([[1]]), i32([2]))),
    ("accept", binding.ATTN_ERR_SHAPE, lambda c: binding.kv_accept(c, i32([0, 400]), i32([[1]]), i32([1]))),
]


def new(c, n):
    x = torch.zeros(n, c.Hkv, c.D, dtype=c.k.dtype, device="cuda")
    return x, x


@pytest.mark.parametrize("case", range(len(BAD)), ids=lambda i: f"{BAD[i][0]}{i}")
def test_wrong_lists_change_nothing_and_are_reported(case):
    _, want, call = BAD[case]
    c = build([40, 33, 16], 16, 2, 64, "f16", 2, n_rows=6)
    m = Model(c)
    call(c)
    assert status() == want
    if BAD[case][0] == "extend" and case == 0:
        m.extend([0], [1])  # the other sequence of the list is served
    m.same(c)


def test_the_same_sequence_twice():
    c = build([40, 33], 16, 2, 64, "f16", n_rows=6)
    m = Model(c)
    binding.kv_extend(c, i32([5, 20]), i32([1, 1]))
    m.extend([1], [5])
    m.same(c)
    assert status() == binding.ATTN_ERR_SHAPE
    binding.kv_fork(c, i32([0, 1]), i32([3, 3]))
    m.fork([0], [3])
    m.same(c)
    assert status() == binding.ATTN_ERR_SHAPE


def test_the_same_sequence_twice_in_append_accept_and_free():
    """The first entry of a list stands; the others are refused (or, freeing, do nothing more)."""
    c = build([40, 33], 16, 2, 64, "f16", n_rows=6)
    x = torch.randn(9, 2, 64, device="cuda").to(DT["f16"])
    m = Model(c)
    seqs, cu = [0, 1, 0, 1], [0, 3, 5, 8, 9]
    binding.kv_append(c, x, x, i32(cu), i32(seqs))
    m.append(0, seqs[:2], x, x, [3, 2])
    assert status() == binding.ATTN_ERR_SHAPE
    m.same(c)
    path = [[1, 2, 3], [0, 2, 3], [0, 1, 2], [2, 3, 3]]
    cu = [0, 5, 9, 14, 18]
    binding.kv_accept(c, i32(cu), i32(path), i32([3, 3, 3, 2]), i32(seqs))
    m.accept(seqs[:2], [5, 4], path[:2])
    assert status() == binding.ATTN_ERR_SHAPE
    m.same(c)
    binding.kv_free(c, i32([1, 0, 1]))
    m.free([1, 0])
    assert status() == binding.ATTN_OK
    m.same(c)


def test_one_token_of_any_row_stride():
    """The row stride of a single token, and the head stride of a single head, are not looked at."""
    c = build([33], 16, 1, 64, "f16", n_rows=2)
    m = Model(c)
    x = torch.randn(64, device="cuda").to(DT["f16"])
    one = x.as_strided((1, 1, 64), (3, 5, 1))
    binding.kv_append(c, one, one, i32([0, 1]), i32([0]))
    m.append(0, [0], one, one, [1])
    assert status() == binding.ATTN_OK
    m.same(c)


def test_shared_and_missing_pages_are_not_written():
    page = 16
    c = build([2 * page, 5], page, 1, 64, "f16", 1, n_rows=6)
    binding.kv_fork(c, i32([0]), i32([2]))  # both pages shared
    m = Model(c)
    x = torch.ones(4, 1, 64, dtype=DT["f16"], device="cuda")
    binding.kv_append(c, x, x, i32([0, 4]), i32([0]))  # the last four rows lie in a shared page
    assert status() == binding.ATTN_ERR_PAGE
    m.same(c)
    binding.kv_accept(c, i32([0, 4]), i32([[1, 2]]), i32([2]), i32([2]))
    assert status() == binding.ATTN_ERR_PAGE
    m.same(c)
    c.table[1, 0] = -1
    m = Model(c)
    binding.kv_append(c, x, x, i32([0, 4]), i32([1]))
    assert status() == binding.ATTN_ERR_PAGE
    m.same(c)


def test_captured_step_replays():
    """Extend, append and accept captured once and replayed: state goes on from replay to replay."""
    page, T = 16, 6
    c = build([30, 9, 47], page, 2, 64, "bf16", 2, extra_pages=20, width=12)
    m = Model(c)
    n_new, cu = i32([T] * 3), offsets([T] * 3)
    path, taken = i32([[0, 2, 5]] * 3), i32([3, 1, 2])
    k_new = torch.randn(3 * T, 2, 64, device="cuda").to(torch.bfloat16)
    v_new = torch.randn(3 * T, 2, 64, device="cuda").to(torch.bfloat16)

    def step():
        binding.kv_extend(c, n_new)
        for layer in range(2):
            binding.kv_append(c, k_new, v_new, cu, layer=layer)
        binding.kv_accept(c, cu, path, taken)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(4):
        taken.copy_(i32([3, i % 4, 2]))
        k_new.normal_()
        g.replay()
        torch.cuda.synchronize()
        m.extend(range(3), [T] * 3)
        for layer in range(2):
            m.append(layer, range(3), k_new, v_new, [T] * 3)
        m.accept(range(3), [T] * 3, [[0, 2, 5][:t] for t in (3, i % 4, 2)])
        m.same(c)
    assert status() == binding.ATTN_OK


def test_pools_past_32_bits():
    """Pages whose elements lie past 2^31: append, fork, compact and copy address them."""
    page, Hkv, D = 256, 8, 128
    n_pages = (1 << 31) // (page * Hkv * D) + 4
    c = binding.KVPages.empty(1, n_pages, Hkv, page, D, 4, 4, torch.bfloat16)
    c.refs.fill_(1)
    c.refs[n_pages - 3:] = 0
    binding.kv_extend(c, i32([page + 100]), i32([1]))
    assert c.table[1].tolist() == [n_pages - 3, n_pages - 2, -1, -1]
    x = torch.randn(page + 100, Hkv, D, device="cuda").to(torch.bfloat16)
    binding.kv_append(c, x, -x, offsets([page + 100]), i32([1]))
    binding.kv_fork(c, i32([1]), i32([2]))
    assert c.table[2].tolist() == [n_pages - 3, n_pages - 1, -1, -1]
    for s in (1, 2):
        at = c.table[s, :2].long()
        got = torch.cat([c.k[0, at[0]].transpose(0, 1), c.k[0, at[1], :, :100].transpose(0, 1)])
        assert torch.equal(got, x)
        got = torch.cat([c.v[0, at[0]].transpose(0, 1), c.v[0, at[1], :, :100].transpose(0, 1)])
        assert torch.equal(got, -x)
    c.refs[:n_pages - 3] = 0
    c.refs[5] = 1
    assert int(binding.kv_compact(c)) == 4  # pages 5, n - 3, n - 2, n - 1 become 0 .. 3
    assert c.table[1].tolist() == [1, 2, -1, -1] and c.table[2].tolist() == [1, 3, -1, -1]
    assert torch.equal(torch.cat([c.k[0, 1].transpose(0, 1), c.k[0, 2, :, :100].transpose(0, 1)]), x)
    binding.kv_copy(c, i32([0]), i32([n_pages - 1]))
    assert torch.equal(c.v[0, n_pages - 1], c.v[0, 0])
    assert status() == binding.ATTN_OK
