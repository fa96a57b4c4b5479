"""Refusals of the packed and paged entry points that need no GPU: every call below fails its
checks, or has nothing to do, before a device is touched."""
import ctypes

import pytest
import torch

from gqa_attention_forward_gb300 import binding, build

P = 0x10000  # an aligned address that is never dereferenced
OK, NULL, SHAPE, HEADDIM, DTYPE, ALIGN, NODEVICE, SCRATCH = 0, 1, 2, 3, 4, 5, 8, 9


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return binding.load()


def no_gpu():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present; this checks the no-device path")


def varlen(**over):
    a = dict(q=P, k=P, v=P, o=P, lse=None, cu_q=P, cu_k=None, n=3, tq=100, tk=100, Hq=4, Hkv=2, D=128,
             strides=None, scale=0.1, causal=1, dtype=1)
    a.update(over)
    return binding.attn_fwd_varlen(a["q"], a["k"], a["v"], a["o"], a["lse"], a["cu_q"], a["cu_k"], a["n"], a["tq"],
                                   a["tk"], a["Hq"], a["Hkv"], a["D"], a["strides"], a["scale"], a["causal"],
                                   a["dtype"], None)


GOOD = [512, 128, 256, 128, 256, 128, 512, 128]


def strides(**at):
    s = list(GOOD)
    for i, x in at.items():
        s[int(i[1:])] = x
    return s


@pytest.mark.parametrize("args,code", [
    (dict(n=-1), SHAPE), (dict(tq=-1), SHAPE), (dict(tk=-1), SHAPE), (dict(Hq=5), SHAPE), (dict(Hkv=0), SHAPE),
    (dict(scale=0.0), SHAPE), (dict(scale=float("nan")), SHAPE), (dict(D=96), HEADDIM), (dict(dtype=2), DTYPE),
    (dict(tk=99), SHAPE),                       # cu_k missing although the keys differ
    (dict(q=0), NULL), (dict(o=0), NULL), (dict(cu_q=0), NULL), (dict(k=0), NULL), (dict(v=0), NULL),
    (dict(q=P + 8), ALIGN), (dict(v=P + 2), ALIGN), (dict(o=P + 4), ALIGN), (dict(lse=P + 2), ALIGN),
    (dict(cu_q=P + 1), ALIGN), (dict(cu_k=P + 2), ALIGN),
    (dict(strides=strides(_0=508)), SHAPE),     # no multiple of 8
    (dict(strides=strides(_1=64)), SHAPE),      # heads overlap
    (dict(strides=strides(_0=384)), SHAPE),     # rows overlap
    (dict(strides=strides(_2=0)), SHAPE),
    (dict(strides=strides(_4=-256)), SHAPE),
    (dict(strides=strides(_6=1 << 40)), SHAPE),
    (dict(strides=strides(_6=520)), SHAPE),     # 520 is no multiple of 128
    (dict(tq=65535 * 128 + 1, tk=65535 * 128 + 1), SHAPE),
    (dict(Hq=1 << 20, Hkv=1 << 20, tq=1 << 22, tk=1 << 22), SHAPE),
])
def test_varlen_argument_errors(args, code):
    assert varlen(**args) == code


@pytest.mark.parametrize("args", [dict(n=0), dict(tq=0, tk=0), dict(Hq=0)])
def test_varlen_empty(args):
    assert varlen(q=None, k=None, v=None, o=None, cu_q=None, **args) == OK


def test_varlen_reaches_the_device_check():
    no_gpu()
    assert varlen() == NODEVICE
    assert varlen(strides=GOOD) == NODEVICE
    assert varlen(strides=[128, 12800, 128, 12800, 128, 12800, 128, 12800]) == NODEVICE  # [heads, rows, D]
    assert varlen(strides=[1024, 128] * 4) == NODEVICE  # cut from one projection
    assert varlen(tk=0, cu_k=P, k=None, v=None) == NODEVICE
    assert varlen(tq=1, tk=1, strides=[8, 128, 3, 128, 0, 128, 1, 128]) == NODEVICE  # one row: its stride is nothing


def cache(**over):
    a = dict(k=P, v=P, table=P, lens=P, refs=P, scratch=P, n_layers=2, n_pages=10, page=16, Hkv=2, D=128, n_rows=4,
             table_width=5, dtype=1)
    a.update(over)
    return binding.KVCache(*(a[n] for n, _ in binding.KVCache._fields_))


CALLS = {
    "extend": lambda c, n=2, **k: binding.attn_kv_extend(c, k.get("seqs"), k.get("n_new", P), n),
    "append": lambda c, n=2, **k: binding.attn_kv_append(c, k.get("layer", 0), k.get("k_new", P), k.get("v_new", P),
                                                         k.get("strides"), k.get("cu", P), k.get("seqs"), n,
                                                         k.get("total", 7)),
    "accept": lambda c, n=2, **k: binding.attn_kv_accept(c, k.get("cu", P), k.get("seqs"), k.get("path", P),
                                                         k.get("width", 3), k.get("taken", P), n),
    "copy": lambda c, n=2, **k: binding.attn_kv_copy(c, k.get("src", P), k.get("dst", P), n),
    "fork": lambda c, n=2, **k: binding.attn_kv_fork(c, k.get("parents", P), k.get("children", P), n),
    "free": lambda c, n=2, **k: binding.attn_kv_free(c, k.get("seqs", P), n),
    "tree": lambda c, n=2, **k: binding.attn_fwd_tree(k.get("q", P), c, k.get("layer", 0), k.get("o", P), k.get("lse"),
                                                      k.get("cu", P), k.get("seqs"), k.get("parents"), n,
                                                      k.get("total", 9), k.get("Hq", 8), k.get("strides"),
                                                      k.get("scale", 0.1), k.get("ws", P), k.get("bytes", 1 << 40)),
}


@pytest.mark.parametrize("args,code", [
    (dict(n_layers=0), SHAPE), (dict(n_pages=0), SHAPE), (dict(Hkv=0), SHAPE), (dict(n_rows=0), SHAPE),
    (dict(table_width=0), SHAPE), (dict(page=8), SHAPE), (dict(page=48), SHAPE), (dict(page=8192), SHAPE),
    (dict(D=96), HEADDIM), (dict(dtype=5), DTYPE), (dict(n_pages=1 << 30), SHAPE), (dict(table_width=1 << 27), SHAPE),
    (dict(n_rows=1 << 30), SHAPE), (dict(n_layers=1 << 20), SHAPE),
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(table=None), NULL), (dict(lens=None), NULL),
    (dict(refs=None), NULL), (dict(scratch=None), NULL),
    (dict(k=P + 8), ALIGN), (dict(table=P + 2), ALIGN), (dict(refs=P + 1), ALIGN),
])
@pytest.mark.parametrize("call", sorted(CALLS))
def test_cache_description_errors(call, args, code):
    assert CALLS[call](cache(**args)) == code


@pytest.mark.parametrize("call", sorted(CALLS))
def test_cache_calls_without_work_and_without_a_cache(call):
    assert CALLS[call](None) == NULL
    assert CALLS[call](cache(), n=0) == OK
    assert CALLS[call](cache(), n=-1) == SHAPE


@pytest.mark.parametrize("call,args,code", [
    ("append", dict(layer=2), SHAPE), ("append", dict(layer=-1), SHAPE), ("append", dict(total=-1), SHAPE),
    ("append", dict(total=0, k_new=None), OK), ("accept", dict(width=0), SHAPE),
    ("tree", dict(layer=2), SHAPE), ("tree", dict(Hq=9), SHAPE), ("tree", dict(Hq=2 * 129), SHAPE),
    ("tree", dict(scale=-1.0), SHAPE), ("tree", dict(total=-1), SHAPE), ("tree", dict(n=5), SHAPE),
    ("tree", dict(q=None), NULL), ("tree", dict(o=None), NULL), ("tree", dict(cu=None), NULL),
    ("tree", dict(ws=None), NULL), ("tree", dict(q=P + 8), ALIGN), ("tree", dict(ws=P + 8), ALIGN),
    ("tree", dict(parents=P + 2), ALIGN), ("tree", dict(lse=P + 1), ALIGN),
    ("tree", dict(strides=[128, 9 * 128, 1024, 128]), SHAPE),   # heads outside rows
    ("tree", dict(strides=[1024, 100, 1024, 128]), SHAPE),
    ("tree", dict(strides=[1024, 128, 512, 128]), SHAPE),
    ("tree", dict(total=0, q=None), OK), ("tree", dict(Hq=0, q=None), OK),
])
def test_call_argument_errors(call, args, code):
    assert CALLS[call](cache(), **args) == code


@pytest.mark.parametrize("call,args,code", [
    ("extend", dict(n_new=None), NULL), ("extend", dict(n=5), SHAPE), ("extend", dict(seqs=P + 1), ALIGN),
    ("append", dict(k_new=None), NULL), ("append", dict(cu=None), NULL), ("append", dict(v_new=P + 8), ALIGN),
    ("append", dict(strides=[256, 128, 256, 100]), SHAPE), ("append", dict(strides=[256, 128, -256, 128]), SHAPE),
    ("accept", dict(path=None), NULL), ("accept", dict(taken=P + 2), ALIGN), ("accept", dict(n=5), SHAPE),
    ("copy", dict(dst=None), NULL), ("copy", dict(src=P + 2), ALIGN),
    ("fork", dict(children=None), NULL), ("fork", dict(n=5), SHAPE), ("free", dict(seqs=None), NULL),
])
def test_list_errors(call, args, code):
    assert CALLS[call](cache(), **args) == code


@pytest.mark.parametrize("call", sorted(CALLS))
def test_good_calls_reach_the_device_check(call):
    no_gpu()
    assert CALLS[call](cache()) == NODEVICE
    assert binding.attn_kv_compact(cache(), None) == NODEVICE
    assert binding.attn_kv_compact(cache(), P + 2) == ALIGN


def test_size_queries():
    st, n = binding.attn_kv_scratch(10, 4)
    assert st == OK and n >= 4 * (2 * 10 + 5 * 4)
    assert binding.attn_kv_scratch(0, 4) == (SHAPE, 0)
    assert binding.attn_fwd_tree_workspace(-1, 128) == (SHAPE, 0)
    assert binding.attn_fwd_tree_workspace(3, 80) == (HEADDIM, 0)
    assert binding.load().attn_kv_scratch(1, 1, None) == NULL
    assert binding.load().attn_fwd_tree_workspace(1, 64, None) == NULL
    assert ctypes.sizeof(binding.KVCache) == 6 * 8 + 8 * 4


def test_python_calls_check_their_tensors():
    bf, i32 = torch.bfloat16, torch.int32
    q, k = torch.zeros(5, 4, 64, dtype=bf), torch.zeros(5, 2, 64, dtype=bf)
    cu = torch.tensor([0, 5], dtype=i32)
    for bad in (
        lambda: binding.attention_varlen(q[0], k, k, cu),
        lambda: binding.attention_varlen(q.transpose(1, 2), k, k, cu),
        lambda: binding.attention_varlen(q, k, k[:4], cu),
        lambda: binding.attention_varlen(q, k[:, :, :32], k[:, :, :32], cu),
        lambda: binding.attention_varlen(q, k.half(), k, cu),
        lambda: binding.attention_varlen(q, k, k, cu.long()),
        lambda: binding.attention_varlen(q, k, k, cu[:0]),
        lambda: binding.attention_varlen(q, k, k, cu, cu[:1]),
        lambda: binding.attention_varlen(q, k, k, cu, out=q[:4]),
        lambda: binding.attention_varlen(q, k, k, cu, out=q.float()),
        lambda: binding.attention_varlen(q, k, k, cu, lse_out=torch.zeros(5, 4)),
    ):
        with pytest.raises(ValueError):
            bad()
    pool = torch.zeros(1, 3, 2, 16, 64, dtype=bf)
    table, lens, refs = torch.full((2, 4), -1, dtype=i32), torch.zeros(2, dtype=i32), torch.zeros(3, dtype=i32)
    for bad in (
        lambda: binding.KVPages(pool[0], pool[0], table, lens, refs),
        lambda: binding.KVPages(pool, pool[:, :2], table, lens, refs),
        lambda: binding.KVPages(pool, pool.half(), table, lens, refs),
        lambda: binding.KVPages(pool, pool, table.long(), lens, refs),
        lambda: binding.KVPages(pool, pool, table, lens[:1], refs),
        lambda: binding.KVPages(pool, pool, table, lens, refs[:2]),
        lambda: binding.KVPages(pool, pool, table, lens, refs, torch.zeros(3, dtype=i32)),
    ):
        with pytest.raises(ValueError):
            bad()
    c = binding.KVPages(pool, pool, table, lens, refs)
    one = torch.zeros(1, dtype=i32)
    for bad in (
        lambda: binding.kv_extend(c, one, lens),
        lambda: binding.kv_extend(c, one.long()),
        lambda: binding.kv_append(c, q, q, cu),
        lambda: binding.kv_append(c, k, k[:3], cu),
        lambda: binding.kv_append(c, k, k, cu, lens),
        lambda: binding.kv_accept(c, cu, one, one),
        lambda: binding.kv_accept(c, cu, one.view(1, 1), lens),
        lambda: binding.kv_copy(c, one, lens),
        lambda: binding.kv_fork(c, one, lens),
        lambda: binding.kv_free(c, table),
        lambda: binding.kv_compact(c, lens),
        lambda: binding.attention_tree(q[:, :3], c, cu),
        lambda: binding.attention_tree(q.half(), c, cu),
        lambda: binding.attention_tree(q, c, cu, parents=lens),
        lambda: binding.attention_tree(q, c, cu, seqs=lens),
        lambda: binding.kv_extend(c, lens),  # everything fits, but nothing is on a GPU
        lambda: binding.kv_append(c, k, k, cu),
        lambda: binding.attention_varlen(q, k, k, cu),
    ):
        with pytest.raises(ValueError):
            bad()
