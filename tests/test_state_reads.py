"""Offsets, lists, lengths and tables that earlier calls write while a later call's blocks are
already resident: no kernel reads them by the read-only path, and calls that follow each other
without a pause give what they give one by one."""
import glob
import os
import random
import re

import pytest
import torch

from gqa_attention_forward_gb300 import binding, build
from paged_util import Model
from paged_util import build as build_cache


def test_no_read_only_loads():
    """The read-only path needs data that is constant while the kernel lives; all inputs of these
    kernels may have been written by the call before, during which their blocks can be resident."""
    for f in glob.glob(os.path.join(build.CSRC, "*.cu*")):
        with open(f) as h:
            code = re.sub(r"//[^\n]*", "", h.read())
        assert not re.search(r"__ldg\s*\(|ld\.global\.nc|__restrict__", code), f


@pytest.mark.gpu
@pytest.mark.parametrize("page,ctx", [(16, [40, 700, 3, 0]), (64, [5000, 64, 1])])
def test_calls_without_a_pause(page, ctx):
    """Extend, append, tree attention, accept, fork, free and compaction, 25 times without a
    synchronisation: the bits of the same calls with one after each."""
    Hq, Hkv, D, n = 8, 2, 128, len(ctx)

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    def loop(pause):
        g = torch.Generator(device="cuda")
        g.manual_seed(5)
        rng = random.Random(5)
        c = binding.KVPages.empty(1, 800, Hkv, page, D, 2 * n, 400, torch.bfloat16)
        c.k.zero_()
        c.v.zero_()

        def rows(m, heads):
            return torch.randn((m, heads, D), generator=g, device="cuda").to(torch.bfloat16)

        steps = [(i32(ctx), i32([0] + torch.tensor(ctx).cumsum(0).tolist()), rows(sum(ctx), Hkv), rows(sum(ctx), Hkv),
                  None, None, None, None)]
        for _ in range(25):
            T = [rng.randint(1, 9) for _ in range(n)]
            par = [t for size in T for t in [-1] + [rng.randint(-1, i - 1) for i in range(1, size)]]
            path = [sorted(rng.sample(range(t), rng.randint(1, t))) for t in T]
            steps.append((i32(T), i32([0] + torch.tensor(T).cumsum(0).tolist()), rows(sum(T), Hkv), rows(sum(T), Hkv),
                          rows(sum(T), Hq), i32(par), i32([x + [-1] * (9 - len(x)) for x in path]),
                          i32([len(x) for x in path])))
        old, new = i32(list(range(n))), i32(list(range(n, 2 * n)))
        torch.cuda.synchronize()
        outs = []

        def after(x=None):
            if pause:
                torch.cuda.synchronize()
            return x

        for T, cu, k, v, q, par, path, taken in steps:
            after(binding.kv_extend(c, T, old))
            after(binding.kv_append(c, k, v, cu, old))
            if q is None:
                continue
            outs += after(binding.attention_tree(q, c, cu, seqs=old, parents=par))
            after(binding.kv_accept(c, cu, path, taken, old))
            after(binding.kv_fork(c, old, new))
            after(binding.kv_free(c, old))
            outs.append(after(binding.kv_compact(c)))
            old, new = new, old
        torch.cuda.synchronize()
        assert binding.attn_last_device_error(torch.cuda.current_stream()) == binding.ATTN_OK
        return outs + [c.lens, c.table, c.refs, c.k, c.v]

    for a, b in zip(loop(True), loop(False)):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_captured_fork_free_and_compaction():
    """A beam step captured once and replayed: the losers are freed, the winners forked into their
    place, the pool made dense; each replay goes on from the state of the one before."""
    page = 16
    c = build_cache([70, 33, 48, 5, 90], page, 2, 64, "bf16", 2, extra_pages=40, n_rows=8)
    m = Model(c)

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    losers, winners = i32([3, 4]), i32([0, 1])
    live = torch.zeros(1, dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        binding.kv_free(c, losers)
        binding.kv_fork(c, winners, losers)
        binding.kv_compact(c, live)
    for lose, win in (([3, 4], [0, 1]), ([0, 1], [2, 2]), ([2, 7], [4, 1]), ([4, 0], [3, 7])):
        losers.copy_(i32(lose))
        winners.copy_(i32(win))
        g.replay()
        torch.cuda.synchronize()
        m.free(lose)
        m.fork(win, lose)
        assert int(live) == m.compact()
        m.same(c)
        m.consistent()
    assert binding.attn_last_device_error(torch.cuda.current_stream()) == binding.ATTN_OK
