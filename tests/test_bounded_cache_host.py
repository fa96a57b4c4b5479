"""Refusals of the window, weighing and eviction entry points that need no GPU: every call below
fails its checks, or has nothing to do, before a device is touched."""
import pytest
import torch

from gqa_attention_forward_gb300 import binding, build
from test_packed_paged_host import ALIGN, DTYPE, HEADDIM, NODEVICE, NULL, OK, P, SHAPE, cache, no_gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return binding.load()


def varlen(**over):
    a = dict(q=P, k=P, v=P, o=P, lse=None, cu_q=P, cu_k=None, n=3, tq=100, tk=100, Hq=4, Hkv=2, D=128, strides=None,
             scale=0.1, window=10, sinks=4, dtype=1)
    a.update(over)
    return binding.attn_fwd_varlen_window(*a.values())


def tree(c, n=2, **k):
    return binding.attn_fwd_tree_window(k.get("q", P), c, k.get("layer", 0), k.get("o", P), k.get("lse"), k.get("cu", P),
                                        k.get("seqs"), k.get("parents"), n, k.get("total", 9), k.get("Hq", 8), k.get("strides"),
                                        k.get("scale", 0.1), k.get("window", 10), k.get("sinks", 0), k.get("ws", P),
                                        k.get("bytes", 1 << 40))


def weigh(c, n=2, **k):
    return binding.attn_kv_weigh(c, k.get("layer", 0), k.get("q", P), k.get("lse", P), k.get("weights", P), k.get("cu", P),
                                 k.get("seqs"), n, k.get("total", 9), k.get("Hq", 8), k.get("strides"), k.get("scale", 0.1), 1)


def evict(c, n=2, **k):
    return binding.attn_kv_evict(c, k.get("seqs", P), n, k.get("weights", P), k.get("sinks", 1), k.get("heavy", 2),
                                 k.get("recent", 3))


@pytest.mark.parametrize("args,code", [
    (dict(window=0), SHAPE), (dict(window=-5), SHAPE), (dict(sinks=-1), SHAPE), (dict(n=-1), SHAPE), (dict(Hq=5), SHAPE),
    (dict(tk=99), SHAPE), (dict(scale=0.0), SHAPE), (dict(D=96), HEADDIM), (dict(dtype=2), DTYPE), (dict(q=0), NULL),
    (dict(k=0), NULL), (dict(cu_q=0), NULL), (dict(v=P + 2), ALIGN), (dict(cu_k=P + 2), ALIGN),
    (dict(strides=[508, 128, 256, 128, 256, 128, 512, 128]), SHAPE),
    (dict(n=0), OK), (dict(tq=0, tk=0, q=0, k=0, v=0, o=0), OK), (dict(Hq=0), OK),
])
def test_window_argument_errors(args, code):
    assert varlen(**args) == code


@pytest.mark.parametrize("args,code", [
    (dict(window=0), SHAPE), (dict(window=-1), SHAPE), (dict(sinks=-1), SHAPE), (dict(layer=2), SHAPE), (dict(Hq=7), SHAPE),
    (dict(scale=float("inf")), SHAPE), (dict(q=None), NULL), (dict(ws=None), NULL), (dict(cu=None), NULL), (dict(o=P + 8), ALIGN),
    (dict(parents=P + 2), ALIGN), (dict(n=9), SHAPE), (dict(n=0), OK), (dict(total=0), OK), (dict(n=-1), SHAPE),
])
def test_tree_window_argument_errors(args, code):
    assert tree(cache(), **args) == code


@pytest.mark.parametrize("args,code", [
    (dict(layer=2), SHAPE), (dict(layer=-1), SHAPE), (dict(Hq=7), SHAPE), (dict(Hq=0), SHAPE), (dict(Hq=2 * 129), SHAPE),
    (dict(scale=-1.0), SHAPE), (dict(scale=float("nan")), SHAPE), (dict(total=-1), SHAPE), (dict(n=5), SHAPE), (dict(n=-1), SHAPE),
    (dict(q=None), NULL), (dict(lse=None), NULL), (dict(weights=None), NULL), (dict(cu=None), NULL), (dict(q=P + 8), ALIGN),
    (dict(lse=P + 2), ALIGN), (dict(weights=P + 1), ALIGN), (dict(cu=P + 2), ALIGN), (dict(seqs=P + 2), ALIGN),
    (dict(strides=[1020, 128]), SHAPE), (dict(strides=[512, 128]), SHAPE), (dict(strides=[128, 1280]), SHAPE),
    (dict(n=0), OK), (dict(total=0, q=None), OK),
])
def test_weigh_argument_errors(args, code):
    assert weigh(cache(), **args) == code


@pytest.mark.parametrize("args,code", [
    (dict(sinks=-1), SHAPE), (dict(heavy=-1), SHAPE), (dict(recent=-1), SHAPE), (dict(n=5), SHAPE), (dict(n=-1), SHAPE),
    (dict(weights=None), NULL), (dict(weights=P + 2), ALIGN), (dict(seqs=P + 1), ALIGN), (dict(n=0, weights=None), OK),
])
def test_evict_argument_errors(args, code):
    assert evict(cache(), **args) == code


@pytest.mark.parametrize("call", [tree, weigh, evict])
@pytest.mark.parametrize("args,code", [
    (dict(n_layers=0), SHAPE), (dict(n_pages=0), SHAPE), (dict(page=48), SHAPE), (dict(D=96), HEADDIM), (dict(dtype=5), DTYPE),
    (dict(table_width=1 << 27), SHAPE), (dict(k=None), NULL), (dict(refs=None), NULL), (dict(k=P + 8), ALIGN)])
def test_cache_description_errors(call, args, code):
    assert call(cache(**args)) == code
    assert call(None) == NULL


def test_right_arguments_reach_the_device_check():
    no_gpu()
    most = 0x7FFFFFFF
    assert varlen() == varlen(window=1, sinks=0) == varlen(window=most, sinks=most) == NODEVICE
    assert tree(cache()) == tree(cache(), window=most, sinks=most) == NODEVICE
    assert weigh(cache()) == weigh(cache(), seqs=P, strides=[2048, 256]) == NODEVICE
    assert evict(cache()) == evict(cache(), seqs=None) == evict(cache(), heavy=0, weights=None) == NODEVICE
    assert evict(cache(), sinks=most, heavy=most, recent=most) == NODEVICE


def test_binding_checks():
    q = torch.zeros(4, 2, 64, dtype=torch.float16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="need a window"):
        binding.attention_varlen(q, q, q, cu, sinks=4)
    with pytest.raises(ValueError, match="causal"):
        binding.attention_varlen(q, q, q, cu, causal=False, window=4)
    i32 = dict(dtype=torch.int32)
    c = binding.KVPages(torch.zeros(2, 5, 1, 16, 64, dtype=torch.float16), torch.zeros(2, 5, 1, 16, 64, dtype=torch.float16),
                        torch.zeros(3, 2, **i32), torch.zeros(3, **i32), torch.zeros(5, **i32))
    w, lse = c.weights(), torch.zeros(2, 4)
    assert w.shape == (2, 3, 1, 32) and w.dtype == torch.float32 and not bool(w.any())
    for bad in (w[:1], w.double(), w.transpose(1, 2)):
        with pytest.raises(ValueError, match="weights"):
            binding.kv_weigh(c, bad, q, lse, cu)
        with pytest.raises(ValueError, match="weights"):
            binding.kv_evict(c, None, bad, heavy=1)
    with pytest.raises(ValueError, match="lse"):
        binding.kv_weigh(c, w, q, lse[:1], cu)
    with pytest.raises(ValueError, match="q must"):
        binding.kv_weigh(c, w, q[:, :, :32].contiguous(), lse, cu)
    with pytest.raises(ValueError, match="seqs"):
        binding.kv_weigh(c, w, q, lse, cu, seqs=cu)
    with pytest.raises(ValueError, match="CUDA device"):
        binding.kv_weigh(c, w, q, lse, cu)
    with pytest.raises(ValueError, match="CUDA device"):
        binding.kv_evict(c, None, w, heavy=1)
