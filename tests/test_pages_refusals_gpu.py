"""Wrong lists and wrong tables: the page operators report them and leave the sequence, its pages
and the pools as they were."""
import pytest
import torch

from gqa_attention_forward_gb300 import binding
from paged_util import Model, build

pytestmark = pytest.mark.gpu

LOWEST = -2 ** 31


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def status():
    return binding.attn_last_device_error(torch.cuda.current_stream())


@pytest.mark.parametrize("path", [[-1], [-1, 0], [-2, -1], [-5, -3, -1, 0], [LOWEST, -2 * 10 ** 9], [LOWEST, LOWEST + 1, 0, 1],
                                  [0, LOWEST], [-1, -1], [3, -7, -6, 2], [0, 2 ** 31 - 1], [2 ** 31 - 1, LOWEST]])
def test_paths_of_no_tree(path):
    """Paths that ascend, but from before the tree, and others that leave it on either side."""
    c = build([40, 5, 33], 16, 2, 64, "f16", 2, n_rows=6)
    m = Model(c)
    for s in (0, 1, 2):
        binding.kv_accept(c, i32([0, 5]), i32([path]), i32([len(path)]), i32([s]))
        assert status() == binding.ATTN_ERR_SHAPE
        m.same(c)
    # one such sequence does not keep the others from being served
    w = max(3, len(path))
    binding.kv_accept(c, i32([0, 5, 9, 12]), i32([x + [-1] * (w - len(x)) for x in ([1, 4], path, [0, 2])]),
                      i32([2, len(path), 2]), i32([0, 1, 2]))
    assert status() == binding.ATTN_ERR_SHAPE
    m.accept([0, 2], [5, 3], [[1, 4], [0, 2]])
    m.same(c)


@pytest.mark.parametrize("page,length", [(16, 64), (16, 70), (32, 32 * 300 + 5), (128, 1)])
@pytest.mark.parametrize("entry", [-1, LOWEST, 10 ** 6, "n_pages"])
def test_fork_of_a_parent_with_a_bad_page(page, length, entry):
    """A page that is missing or out of range, full or not, first, middle or last: the request is
    refused as a whole and the others of the list are served, in their order."""
    pages = -(-length // page)
    for j in sorted({0, pages // 2, pages - 1}):
        c = build([length, 2 * page + 3, page], page, 2, 64, "f16", 1, extra_pages=5, n_rows=9)
        c.table[0, j] = c.n_pages if entry == "n_pages" else entry
        m = Model(c)
        binding.kv_fork(c, i32([0]), i32([4]))
        assert status() == binding.ATTN_ERR_PAGE
        m.same(c)
        binding.kv_fork(c, i32([1, 0, 2, 0, 1]), i32([5, 4, 6, 3, 7]))
        assert status() == binding.ATTN_ERR_PAGE
        m.fork([1, 2, 1], [5, 6, 7])
        m.same(c)


def test_fork_of_many_parents_of_which_some_are_bad():
    """More requests than the cluster has warps."""
    page, n = 16, 700
    lens = [(37 * i) % 100 for i in range(n)]
    c = build(lens, page, 1, 64, "bf16", extra_pages=n, seed=6, n_rows=2 * n)
    bad = [i for i in range(n) if lens[i] > page and i % 5 == 0]
    for i in bad:
        c.table[i, 0] = -1 if i % 2 else c.n_pages + i
    m = Model(c)
    binding.kv_fork(c, i32(list(range(n))), i32([n + i for i in range(n)]))
    assert status() == binding.ATTN_ERR_PAGE
    good = [i for i in range(n) if i not in bad]
    m.fork(good, [n + i for i in good])
    m.same(c)


def test_fork_of_a_length_past_the_table():
    c = build([40, 20], 16, 2, 64, "f16", n_rows=6)
    for length in (-1, 10 ** 6, 2 ** 31 - 1):
        c.lens[0] = length
        m = Model(c)
        binding.kv_fork(c, i32([0, 1]), i32([4, 5]))
        assert status() == binding.ATTN_ERR_SHAPE
        m.fork([1], [5])
        m.same(c)
        binding.kv_free(c, i32([5]))


@pytest.mark.parametrize("seqs", [None, [0, 1, 2]])
def test_extend_over_a_kept_page_out_of_range(seqs):
    """A sequence ends before pages that it has kept (as after accepting a tree), one of which is
    no page of the pool: refused, the others are served."""
    page = 16
    c = build([100, 20, 90], page, 2, 64, "f16", extra_pages=6, n_rows=5)
    c.lens[0] = 30  # five pages of its seven are kept behind its end
    s = None if seqs is None else i32(seqs)
    for wrong in (c.n_pages, 10 ** 6, 2 ** 31 - 1):
        good = int(c.table[0, 4])
        c.table[0, 4] = wrong
        m = Model(c)
        binding.kv_extend(c, i32([60, 15, 7]), s)
        assert status() == binding.ATTN_ERR_PAGE
        m.extend([1, 2], [15, 7])
        m.same(c)
        binding.kv_extend(c, i32([34, 0, 0]), s)  # up to the page before it: served
        m.extend([0], [34])
        m.same(c)
        assert status() == binding.ATTN_OK
        c.table[0, 4] = good
        c.lens[0] = 30
