"""ctypes binding of libgqa_attn.so (argument marshalling only).

Every step of the attention forward runs inside the library's CUDA kernel;
this module converts Python / torch arguments to the C ABI declared in
``include/gqa_attn.h`` and turns status codes into exceptions.  There is no
fallback: if the library is missing or the device is not sm_103, calls raise.
"""
from __future__ import annotations

import ctypes
import math
import os
import threading

from . import build as _build

ATTN_F16, ATTN_BF16 = 0, 1
STATUS = {0: "ATTN_OK", 1: "ATTN_ERR_NULL", 2: "ATTN_ERR_SHAPE", 3: "ATTN_ERR_HEADDIM",
          4: "ATTN_ERR_DTYPE", 5: "ATTN_ERR_ALIGN", 6: "ATTN_ERR_LAUNCH", 7: "ATTN_ERR_TIMEOUT",
          8: "ATTN_ERR_NODEVICE", 9: "ATTN_ERR_SCRATCH", 10: "ATTN_ERR_PAGE", 11: "ATTN_ERR_POOL"}
ATTN_OK, ATTN_ERR_SHAPE, ATTN_ERR_TIMEOUT, ATTN_ERR_SCRATCH = 0, 2, 7, 9
ATTN_ERR_PAGE, ATTN_ERR_POOL = 10, 11

_lock = threading.Lock()
_lib = None


class AttnError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {STATUS.get(status, status)}")


class KVCache(ctypes.Structure):
    """attn_kv_cache_t: a paged key/value cache as the C entry points take it."""

    _fields_ = ([(n, ctypes.c_void_p) for n in ("k", "v", "table", "lens", "refs", "scratch")]
                + [(n, ctypes.c_int) for n in ("n_layers", "n_pages", "page", "Hkv", "D", "n_rows",
                                               "table_width", "dtype")])


def load(path: str | None = None):
    """Load the built library (no build here: a missing library is an error)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or _build.LIB
        if not os.path.exists(p):
            raise RuntimeError(f"{p} is not built; call gqa_attention_forward_gb300.build.build()")
        lib = ctypes.CDLL(p)
        vp, i = ctypes.c_void_p, ctypes.c_int
        lib.attn_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, ctypes.c_float, i, i, vp]
        lib.attn_fwd.restype = i
        lib.attn_fwd_kv.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, ctypes.c_float, i, i, vp]
        lib.attn_fwd_kv.restype = i
        lib.attn_fwd_decode.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, ctypes.c_float, i, i,
                                        vp, ctypes.c_size_t, vp]
        lib.attn_fwd_decode.restype = i
        lib.attn_fwd_decode_noalloc.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, ctypes.c_float,
                                                i, i, vp]
        lib.attn_fwd_decode_noalloc.restype = i
        lib.attn_fwd_host.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i,
                                      ctypes.c_float, i, i, vp]
        lib.attn_fwd_host.restype = i
        lib.attn_fwd_decode_workspace.argtypes = [i, i, i, i, i, i, ctypes.POINTER(ctypes.c_size_t)]
        lib.attn_fwd_decode_workspace.restype = i
        lib.attn_fwd_kv_split.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, ctypes.c_float, i, i,
                                          vp, ctypes.c_size_t, vp]
        lib.attn_fwd_kv_split.restype = i
        lib.attn_fwd_kv_split_workspace.argtypes = [i, i, i, i, i, i, i, ctypes.POINTER(ctypes.c_size_t)]
        lib.attn_fwd_kv_split_workspace.restype = i
        sz, pc = ctypes.c_size_t, ctypes.POINTER(KVCache)
        lib.attn_fwd_varlen.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, vp,
                                        ctypes.c_float, i, i, vp]
        lib.attn_fwd_varlen.restype = i
        lib.attn_fwd_tree_workspace.argtypes = [i, i, ctypes.POINTER(sz)]
        lib.attn_fwd_tree_workspace.restype = i
        lib.attn_fwd_tree.argtypes = [vp, pc, i, vp, vp, vp, vp, vp, i, i, i, vp, ctypes.c_float, vp,
                                      sz, vp]
        lib.attn_fwd_tree.restype = i
        lib.attn_kv_scratch.argtypes = [i, i, ctypes.POINTER(sz)]
        lib.attn_kv_scratch.restype = i
        lib.attn_kv_extend.argtypes = [pc, vp, vp, i, vp]
        lib.attn_kv_extend.restype = i
        lib.attn_kv_append.argtypes = [pc, i, vp, vp, vp, vp, vp, i, i, vp]
        lib.attn_kv_append.restype = i
        lib.attn_kv_accept.argtypes = [pc, vp, vp, vp, i, vp, i, vp]
        lib.attn_kv_accept.restype = i
        lib.attn_kv_copy.argtypes = [pc, vp, vp, i, vp]
        lib.attn_kv_copy.restype = i
        lib.attn_kv_fork.argtypes = [pc, vp, vp, i, vp]
        lib.attn_kv_fork.restype = i
        lib.attn_kv_free.argtypes = [pc, vp, i, vp]
        lib.attn_kv_free.restype = i
        lib.attn_kv_compact.argtypes = [pc, vp, vp]
        lib.attn_kv_compact.restype = i
        lib.attn_test_force_splits.argtypes = [i]
        lib.attn_test_force_splits.restype = None
        lib.attn_status_str.argtypes = [i]
        lib.attn_status_str.restype = ctypes.c_char_p
        lib.attn_last_device_error.argtypes = [vp]
        lib.attn_last_device_error.restype = i
        lib.attn_last_cuda_error.argtypes = []
        lib.attn_last_cuda_error.restype = ctypes.c_char_p
        lib.attn_version.argtypes = []
        lib.attn_version.restype = i
        lib.attn_test_set_wait_timeout_ns.argtypes = [ctypes.c_ulonglong]
        lib.attn_test_set_wait_timeout_ns.restype = None
        lib.attn_test_inject_stall.argtypes = [i]
        lib.attn_test_inject_stall.restype = None
        lib.attn_test_select_kernel.argtypes = [i]
        lib.attn_test_select_kernel.restype = None
        lib.attn_test_set_item_order.argtypes = [i]
        lib.attn_test_set_item_order.restype = None
        if path is None:
            _lib = lib
        return lib


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _dtype_code(dtype) -> int:
    if isinstance(dtype, int):
        return dtype
    name = str(dtype)
    if name in ("f16", "torch.float16", "float16"):
        return ATTN_F16
    if name in ("bf16", "torch.bfloat16", "bfloat16"):
        return ATTN_BF16
    return -1


def _stream_handle(stream):
    if stream is None:
        return None
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def attn_fwd(q, k, v, o, lse, B, Hq, Hkv, N, D, scale, causal, dtype, stream=None) -> int:
    """The C entry point with the same name; returns its status code."""
    lib = load()
    return lib.attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), int(B), int(Hq), int(Hkv),
                        int(N), int(D), float(scale), int(bool(causal)), _dtype_code(dtype),
                        _stream_handle(stream))


def attn_fwd_kv(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, D, scale, causal, dtype, stream=None) -> int:
    """The C entry point with the same name; returns its status code."""
    lib = load()
    return lib.attn_fwd_kv(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), int(B), int(Hq),
                           int(Hkv), int(Nq), int(Nk), int(D), float(scale), int(bool(causal)),
                           _dtype_code(dtype), _stream_handle(stream))


def attn_fwd_decode(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, D, scale, causal, dtype, workspace,
                    workspace_bytes, stream=None) -> int:
    """The C entry point with the same name; returns its status code."""
    lib = load()
    return lib.attn_fwd_decode(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), int(B), int(Hq),
                               int(Hkv), int(Nq), int(Nk), int(D), float(scale), int(bool(causal)),
                               _dtype_code(dtype), _ptr(workspace), int(workspace_bytes),
                               _stream_handle(stream))


def attn_fwd_kv_split(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, D, scale, causal, dtype, workspace,
                      workspace_bytes, stream=None) -> int:
    """The C entry point with the same name; returns its status code."""
    lib = load()
    return lib.attn_fwd_kv_split(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), int(B), int(Hq),
                                 int(Hkv), int(Nq), int(Nk), int(D), float(scale), int(bool(causal)),
                                 _dtype_code(dtype), _ptr(workspace), int(workspace_bytes),
                                 _stream_handle(stream))


def attn_fwd_kv_split_workspace(B, Hq, Hkv, Nq, Nk, D, causal):
    """(status, bytes) of the C entry point with the same name."""
    n = ctypes.c_size_t(0)
    st = load().attn_fwd_kv_split_workspace(int(B), int(Hq), int(Hkv), int(Nq), int(Nk), int(D),
                                            int(bool(causal)), ctypes.byref(n))
    return st, n.value


def attn_fwd_decode_noalloc(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, D, scale, causal, dtype,
                            stream=None) -> int:
    """The C entry point with the same name; returns its status code."""
    lib = load()
    return lib.attn_fwd_decode_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), int(B),
                                       int(Hq), int(Hkv), int(Nq), int(Nk), int(D), float(scale),
                                       int(bool(causal)), _dtype_code(dtype), _stream_handle(stream))


def attn_fwd_host(q_h, k_h, v_h, o_h, lse_h, q_d, k_d, v_d, o_d, lse_d, B, Hq, Hkv, Nq, Nk, D,
                  scale, causal, dtype, stream=None) -> int:
    """The C entry point with the same name; returns its status code.  Host
    arguments are CPU tensors (pinned for overlap), device arguments CUDA tensors."""
    lib = load()
    return lib.attn_fwd_host(_ptr(q_h), _ptr(k_h), _ptr(v_h), _ptr(o_h), _ptr(lse_h), _ptr(q_d),
                             _ptr(k_d), _ptr(v_d), _ptr(o_d), _ptr(lse_d), int(B), int(Hq), int(Hkv),
                             int(Nq), int(Nk), int(D), float(scale), int(bool(causal)),
                             _dtype_code(dtype), _stream_handle(stream))


def attn_fwd_decode_workspace(B, Hq, Hkv, Nq, Nk, D):
    """(status, bytes) of the C entry point with the same name."""
    n = ctypes.c_size_t(0)
    st = load().attn_fwd_decode_workspace(int(B), int(Hq), int(Hkv), int(Nq), int(Nk), int(D),
                                          ctypes.byref(n))
    return st, n.value


def attention_decode(q, k, v, causal: bool = True, scale: float | None = None,
                     with_lse: bool = True, workspace=None, out=None, lse_out=None, stream=None):
    """attn_fwd_decode for torch CUDA tensors q [B,Hq,Nq,D], k/v [B,Hkv,Nk,D].

    ``workspace``: a uint8 CUDA tensor, or None to let torch allocate the size
    attn_fwd_decode_workspace asks for.  Returns (o, lse) without waiting."""
    import torch

    B, Hq, Nq, D = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    for t in (q, k, v):
        if not t.is_contiguous():
            raise ValueError("q, k, v must be contiguous [B, H, N, D]")
    o = out if out is not None else torch.empty_like(q)
    lse = None
    if with_lse:
        lse = lse_out if lse_out is not None else torch.empty((B, Hq, Nq), dtype=torch.float32,
                                                              device=q.device)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if workspace is None:
        st, nbytes = attn_fwd_decode_workspace(B, Hq, Hkv, Nq, Nk, D)
        if st != ATTN_OK:
            raise AttnError(st, "attn_fwd_decode_workspace")
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=q.device)
    if stream is None:
        stream = torch.cuda.current_stream(q.device)
    st = attn_fwd_decode(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, D, scale, causal, q.dtype,
                         workspace, workspace.numel(), stream)
    if st != ATTN_OK:
        raise AttnError(st, f"attn_fwd_decode ({attn_last_cuda_error()})")
    return o, lse


def attention_split(q, k, v, causal: bool = True, scale: float | None = None, with_lse: bool = True,
                    workspace=None, out=None, lse_out=None, stream=None):
    """attn_fwd_kv_split for torch CUDA tensors q [B,Hq,Nq,D], k/v [B,Hkv,Nk,D].

    ``workspace``: a uint8 CUDA tensor (256-byte aligned, as torch allocates), or
    None to let torch allocate the size attn_fwd_kv_split_workspace asks for.
    Returns (o, lse) without waiting."""
    import torch

    B, Hq, Nq, D = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    for t in (q, k, v):
        if not t.is_contiguous():
            raise ValueError("q, k, v must be contiguous [B, H, N, D]")
    o = out if out is not None else torch.empty_like(q)
    lse = None
    if with_lse:
        lse = lse_out if lse_out is not None else torch.empty((B, Hq, Nq), dtype=torch.float32,
                                                              device=q.device)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if workspace is None:
        st, nbytes = attn_fwd_kv_split_workspace(B, Hq, Hkv, Nq, Nk, D, causal)
        if st != ATTN_OK:
            raise AttnError(st, "attn_fwd_kv_split_workspace")
        workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=q.device)
    if stream is None:
        stream = torch.cuda.current_stream(q.device)
    st = attn_fwd_kv_split(q, k, v, o, lse, B, Hq, Hkv, Nq, Nk, D, scale, causal, q.dtype,
                           workspace, workspace.numel(), stream)
    if st != ATTN_OK:
        raise AttnError(st, f"attn_fwd_kv_split ({attn_last_cuda_error()})")
    return o, lse


def attn_status_str(status: int) -> str:
    return load().attn_status_str(int(status)).decode()


def attn_last_device_error(stream=None) -> int:
    return load().attn_last_device_error(_stream_handle(stream))


def attn_last_cuda_error() -> str:
    return load().attn_last_cuda_error().decode()


def attn_version() -> int:
    return load().attn_version()


def attention(q, k, v, causal: bool = True, scale: float | None = None, with_lse: bool = True,
              out=None, lse_out=None, stream=None):
    """O (and LSE) for torch CUDA tensors q [B,Hq,Nq,D], k/v [B,Hkv,Nk,D] (fp16 or bf16).

    With Nq != Nk the causal mask is bottom-right aligned (attn_fwd_kv).  torch
    allocates the outputs; the library computes them.  Launches on ``stream``
    (default: torch's current stream) and returns without waiting."""
    import torch

    B, Hq, N, D = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    for t in (q, k, v):
        if not t.is_contiguous():
            raise ValueError("q, k, v must be contiguous [B, H, N, D]")
    o = out if out is not None else torch.empty_like(q)
    lse = None
    if with_lse:
        lse = lse_out if lse_out is not None else torch.empty((B, Hq, N), dtype=torch.float32,
                                                              device=q.device)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if stream is None:
        stream = torch.cuda.current_stream(q.device)
    if Nk == N:
        st = attn_fwd(q, k, v, o, lse, B, Hq, Hkv, N, D, scale, causal, q.dtype, stream)
    else:
        st = attn_fwd_kv(q, k, v, o, lse, B, Hq, Hkv, N, Nk, D, scale, causal, q.dtype, stream)
    if st != ATTN_OK:
        raise AttnError(st, f"attn_fwd ({attn_last_cuda_error()})")
    return o, lse


# ------------------------------------------------------------------ packed sequences
_Strides4, _Strides8 = ctypes.c_longlong * 4, ctypes.c_longlong * 8


def _strides(values):
    """Element strides as the C entry points take them (None stays None)."""
    return None if values is None else (ctypes.c_longlong * len(values))(*values)


def attn_fwd_varlen(q, k, v, o, lse, cu_q, cu_k, n_seqs, total_q, total_k, Hq, Hkv, D, strides, scale,
                    causal, dtype, stream=None) -> int:
    """The C entry point with the same name; returns its status code.  ``strides``:
    None or 8 element strides."""
    return load().attn_fwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(cu_q), _ptr(cu_k),
                                  int(n_seqs), int(total_q), int(total_k), int(Hq), int(Hkv), int(D),
                                  _strides(strides), float(scale), int(bool(causal)), _dtype_code(dtype),
                                  _stream_handle(stream))


_torch_module = None


def _torch():
    """torch, imported on first use."""
    global _torch_module
    if _torch_module is None:
        import torch

        _torch_module = torch
    return _torch_module


# What the calls below do per call on the host is kept short: with one short prompt or one
# draft tree the launch and this code take longer than the kernel.
def _rows(t, name):
    """(rows, heads, D) of a packed tensor and its strides."""
    s = t.stride()
    if len(s) != 3 or s[2] != 1:
        raise ValueError(f"{name} must be [tokens, heads, D] with the last axis contiguous")
    return t.shape, s


def _ints(t, name, dev, shape=None):
    """Checks an int32 index tensor on device number ``dev`` (-1: the host)."""
    if t.dtype != _torch().int32 or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor on the device of the others")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    return t


def _same(t, name, dtype, dev):
    if t.dtype != dtype or t.get_device() != dev:
        raise ValueError(f"{name} must be {dtype} on the device of the others")


def _run(what, dev, stream, entry, *args):
    """entry(*args, stream handle) with device ``dev`` current; raises AttnError unless it succeeds."""
    torch = _torch()
    if dev < 0:
        raise ValueError(f"{what}: the tensors must be on a CUDA device")
    handle = torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream_handle(stream)
    if torch._C._cuda_getDevice() == dev:
        st = entry(*args, handle)
    else:
        with torch.cuda.device(dev):
            st = entry(*args, handle)
    if st != ATTN_OK:
        raise AttnError(st, f"{what} ({attn_last_cuda_error()})")


def _new(q, shape, dtype, stream):
    """A new tensor beside q, in memory of ``stream`` (None: the current one), which nothing
    earlier still uses there; it is kept, too, for what the current stream does with it."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=q.device)
    if isinstance(stream, int):  # 0 to 2: the default stream's handles
        stream = (torch.cuda.default_stream(q.device) if stream < 3
                  else torch.cuda.ExternalStream(stream, device=q.device))
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=q.device)
    t.record_stream(torch.cuda.current_stream(q.device))
    return t


def _outputs(q, dev, Hq, total, with_lse, out, lse_out, stream):
    """The output tensors: new ones, or the given ones checked."""
    torch = _torch()
    if out is None:
        out = _new(q, q.shape, q.dtype, stream)
    else:
        _same(out, "out", q.dtype, dev)
        if out.shape != q.shape:
            raise ValueError(f"out must have shape {tuple(q.shape)}")
    if not with_lse:
        return out, None
    if lse_out is None:
        return out, _new(q, (Hq, total), torch.float32, stream)
    _same(lse_out, "lse_out", torch.float32, dev)
    if lse_out.shape != (Hq, total) or not lse_out.is_contiguous():
        raise ValueError(f"lse_out must be contiguous [{Hq}, {total}]")
    return out, lse_out


def attention_varlen(q, k, v, cu_q, cu_k=None, causal: bool = True, scale: float | None = None,
                     with_lse: bool = True, out=None, lse_out=None, stream=None):
    """attn_fwd_varlen for torch CUDA tensors q [total_q,Hq,D], k/v [total_k,Hkv,D] (any row and
    head strides that the C entry point takes, e.g. heads cut from one projection's output).

    ``cu_q`` (and ``cu_k`` where the keys' offsets differ): int32 [n_seqs + 1] offsets on the
    device, never read by the host.  Returns (o [total_q,Hq,D], lse [Hq,total_q]) without waiting;
    rows behind the last sequence are not written."""
    shape, sq = _rows(q, "q")
    kshape, sk = _rows(k, "k")
    vshape, sv = _rows(v, "v")
    total_q, Hq, D = shape
    total_k, Hkv, Dk = kshape
    if vshape != kshape or Dk != D:
        raise ValueError("k and v must have one shape [total_k, Hkv, D] with q's D")
    dev, dtype = q.get_device(), q.dtype
    _same(k, "k", dtype, dev)
    _same(v, "v", dtype, dev)
    _ints(cu_q, "cu_q", dev)
    if cu_q.dim() != 1 or cu_q.numel() < 1:
        raise ValueError("cu_q must hold n_seqs + 1 offsets")
    if cu_k is not None:
        _ints(cu_k, "cu_k", dev, cu_q.shape)
    o, lse = _outputs(q, dev, Hq, total_q, with_lse, out, lse_out, stream)
    so = o.stride()
    if so[2] != 1:
        raise ValueError("out must have its last axis contiguous")
    _run("attn_fwd_varlen", dev, stream, load().attn_fwd_varlen, q.data_ptr(), k.data_ptr(), v.data_ptr(),
         o.data_ptr(), _ptr(lse), cu_q.data_ptr(), _ptr(cu_k), cu_q.numel() - 1, total_q, total_k, Hq, Hkv, D,
         _Strides8(sq[0], sq[1], sk[0], sk[1], sv[0], sv[1], so[0], so[1]),
         D ** -0.5 if scale is None else scale, 1 if causal else 0, _dtype_code(dtype))
    return o, lse


# ------------------------------------------------------------------ paged cache
def attn_kv_scratch(n_pages, n_rows):
    """(status, bytes) of the C entry point with the same name."""
    n = ctypes.c_size_t(0)
    st = load().attn_kv_scratch(int(n_pages), int(n_rows), ctypes.byref(n))
    return st, n.value


class KVPages:
    """A paged key/value cache over torch CUDA tensors (attn_kv_cache_t).

    k, v   [n_layers, n_pages, Hkv, page, D] pools (fp16 or bf16)
    table  int32 [n_rows, table_width] pages of each sequence, -1 behind the last
    lens   int32 [n_rows] positions of each sequence
    refs   int32 [n_pages] table entries that name the page; 0: free

    The tensors stay the caller's and are changed in place; the object holds them and the
    scratch of the calls.  Calls on one cache must be ordered on the device."""

    def __init__(self, k, v, table, lens, refs, scratch=None):
        import torch

        if k.dim() != 5 or v.shape != k.shape or not (k.is_contiguous() and v.is_contiguous()):
            raise ValueError("k and v must be contiguous [n_layers, n_pages, Hkv, page, D]")
        _same(v, "v", k.dtype, k.get_device())
        n_layers, n_pages, Hkv, page, D = k.shape
        if table.dim() != 2:
            raise ValueError("table must be [n_rows, table_width]")
        dev = k.get_device()
        _ints(table, "table", dev)
        _ints(lens, "lens", dev, (table.shape[0],))
        _ints(refs, "refs", dev, (n_pages,))
        st, nbytes = attn_kv_scratch(n_pages, table.shape[0])
        if st != ATTN_OK:
            raise AttnError(st, "attn_kv_scratch")
        if scratch is None:
            scratch = torch.empty(nbytes // 4, dtype=torch.int32, device=k.device)
        _ints(scratch, "scratch", dev)
        if scratch.numel() * 4 < nbytes:
            raise ValueError(f"scratch must hold {nbytes // 4} ints")
        self.k, self.v, self.table, self.lens, self.refs, self.scratch = k, v, table, lens, refs, scratch
        self.device, self.dev, self.dtype = k.device, dev, k.dtype
        self.n_rows, self.table_width = table.shape
        self.n_layers, self.n_pages, self.Hkv, self.page, self.D = n_layers, n_pages, Hkv, page, D
        self.c = KVCache(_ptr(k), _ptr(v), _ptr(table), _ptr(lens), _ptr(refs), _ptr(scratch), n_layers,
                         n_pages, page, Hkv, D, self.n_rows, self.table_width, _dtype_code(k.dtype))
        self.ref = ctypes.byref(self.c)

    @classmethod
    def empty(cls, n_layers, n_pages, Hkv, page, D, n_rows, table_width, dtype, device="cuda"):
        """A cache without sequences (pool contents undefined)."""
        import torch

        k, v = (torch.empty((n_layers, n_pages, Hkv, page, D), dtype=dtype, device=device) for _ in "kv")
        i32 = dict(dtype=torch.int32, device=device)
        return cls(k, v, torch.full((n_rows, table_width), -1, **i32), torch.zeros(n_rows, **i32),
                   torch.zeros(n_pages, **i32))


def _c(cache):
    """The C structure of a KVPages, or what the caller passes in its place."""
    c = cache.c if isinstance(cache, KVPages) else cache
    return None if c is None else ctypes.byref(c)


def attn_kv_extend(cache, seqs, n_new, n, stream=None) -> int:
    """The C entry point with the same name; returns its status code."""
    return load().attn_kv_extend(_c(cache), _ptr(seqs), _ptr(n_new), int(n), _stream_handle(stream))


def attn_kv_append(cache, layer, k_new, v_new, strides, cu, seqs, n, total, stream=None) -> int:
    """The C entry point with the same name; returns its status code."""
    return load().attn_kv_append(_c(cache), int(layer), _ptr(k_new), _ptr(v_new), _strides(strides), _ptr(cu),
                                 _ptr(seqs), int(n), int(total), _stream_handle(stream))


def attn_kv_accept(cache, cu, seqs, path, path_width, taken, n, stream=None) -> int:
    """The C entry point with the same name; returns its status code."""
    return load().attn_kv_accept(_c(cache), _ptr(cu), _ptr(seqs), _ptr(path), int(path_width), _ptr(taken),
                                 int(n), _stream_handle(stream))


def attn_kv_copy(cache, src, dst, n, stream=None) -> int:
    """The C entry point with the same name; returns its status code."""
    return load().attn_kv_copy(_c(cache), _ptr(src), _ptr(dst), int(n), _stream_handle(stream))


def attn_kv_fork(cache, parents, children, n, stream=None) -> int:
    """The C entry point with the same name; returns its status code."""
    return load().attn_kv_fork(_c(cache), _ptr(parents), _ptr(children), int(n), _stream_handle(stream))


def attn_kv_free(cache, seqs, n, stream=None) -> int:
    """The C entry point with the same name; returns its status code."""
    return load().attn_kv_free(_c(cache), _ptr(seqs), int(n), _stream_handle(stream))


def attn_kv_compact(cache, live, stream=None) -> int:
    """The C entry point with the same name; returns its status code."""
    return load().attn_kv_compact(_c(cache), _ptr(live), _stream_handle(stream))


def attn_fwd_tree_workspace(n_seqs, D):
    """(status, bytes) of the C entry point with the same name."""
    n = ctypes.c_size_t(0)
    st = load().attn_fwd_tree_workspace(int(n_seqs), int(D), ctypes.byref(n))
    return st, n.value


def attn_fwd_tree(q, cache, layer, o, lse, cu, seqs, parents, n_seqs, total_q, Hq, strides, scale, workspace,
                  workspace_bytes, stream=None) -> int:
    """The C entry point with the same name; returns its status code.  ``strides``: None or 4
    element strides."""
    return load().attn_fwd_tree(_ptr(q), _c(cache), int(layer), _ptr(o), _ptr(lse), _ptr(cu), _ptr(seqs),
                                _ptr(parents), int(n_seqs), int(total_q), int(Hq), _strides(strides),
                                float(scale), _ptr(workspace), int(workspace_bytes), _stream_handle(stream))


def _list(t, name, cache, n=None):
    """Checks an int32 list on the cache's device (None is taken); returns its length."""
    if t is None:
        return n
    if t.dim() != 1:
        raise ValueError(f"{name} must be one-dimensional")
    _ints(t, name, cache.dev, None if n is None else (n,))
    return t.shape[0]


def kv_extend(cache, n_new, seqs=None, stream=None):
    """attn_kv_extend: room for n_new[i] more positions of sequence seqs[i] (i, when None)."""
    n = _list(n_new, "n_new", cache)
    _list(seqs, "seqs", cache, n)
    _run("attn_kv_extend", cache.dev, stream, load().attn_kv_extend, cache.ref, _ptr(seqs), n_new.data_ptr(), n)


def kv_append(cache, k_new, v_new, cu, seqs=None, layer: int = 0, stream=None):
    """attn_kv_append: packed rows k_new, v_new [total,Hkv,D] become the last positions of the
    sequences (offsets ``cu`` [n + 1]), whose lens already counts them."""
    shape, sk = _rows(k_new, "k_new")
    vshape, sv = _rows(v_new, "v_new")
    if shape != vshape or shape[1] != cache.Hkv or shape[2] != cache.D:
        raise ValueError("k_new and v_new must be [total, Hkv, D] with the cache's Hkv and D")
    _same(k_new, "k_new", cache.dtype, cache.dev)
    _same(v_new, "v_new", cache.dtype, cache.dev)
    n = _list(cu, "cu", cache) - 1
    _list(seqs, "seqs", cache, n)
    _run("attn_kv_append", cache.dev, stream, load().attn_kv_append, cache.ref, layer, k_new.data_ptr(),
         v_new.data_ptr(), _Strides4(sk[0], sk[1], sv[0], sv[1]), cu.data_ptr(), _ptr(seqs), n, shape[0])


def kv_accept(cache, cu, path, taken, seqs=None, stream=None):
    """attn_kv_accept: of each tree (offsets ``cu``), the tokens path[i, :taken[i]] stay."""
    n = _list(cu, "cu", cache) - 1
    _list(seqs, "seqs", cache, n)
    _list(taken, "taken", cache, n)
    if path.dim() != 2 or path.shape[0] != n:
        raise ValueError("path must be [n, path_width]")
    _ints(path, "path", cache.dev)
    _run("attn_kv_accept", cache.dev, stream, load().attn_kv_accept, cache.ref, cu.data_ptr(), _ptr(seqs),
         path.data_ptr(), path.shape[1], taken.data_ptr(), n)


def kv_copy(cache, src, dst, stream=None):
    """attn_kv_copy: the contents of pages src[i] go to pages dst[i], in every layer."""
    n = _list(src, "src", cache)
    _list(dst, "dst", cache, n)
    _run("attn_kv_copy", cache.dev, stream, load().attn_kv_copy, cache.ref, src.data_ptr(), dst.data_ptr(), n)


def kv_fork(cache, parents, children, stream=None):
    """attn_kv_fork: the empty sequences children[i] become copies of parents[i]."""
    n = _list(parents, "parents", cache)
    _list(children, "children", cache, n)
    _run("attn_kv_fork", cache.dev, stream, load().attn_kv_fork, cache.ref, parents.data_ptr(),
         children.data_ptr(), n)


def kv_free(cache, seqs, stream=None):
    """attn_kv_free: the sequences become empty and give their pages back."""
    n = _list(seqs, "seqs", cache)
    _run("attn_kv_free", cache.dev, stream, load().attn_kv_free, cache.ref, seqs.data_ptr(), n)


def kv_compact(cache, live=None, stream=None):
    """attn_kv_compact: the live pages become pages 0 .. live - 1.  Returns the int32 [1] tensor
    that receives ``live``."""
    if live is None:
        live = _new(cache.lens, (1,), cache.lens.dtype, stream)
    else:
        _ints(live, "live", cache.dev, (1,))
    _run("attn_kv_compact", cache.dev, stream, load().attn_kv_compact, cache.ref, live.data_ptr())
    return live


_tree_bytes = {}  # (device number, sequences, D) -> bytes of attn_fwd_tree_workspace


def attention_tree(q, cache, cu, seqs=None, parents=None, layer: int = 0, scale: float | None = None,
                   with_lse: bool = True, workspace=None, out=None, lse_out=None, stream=None):
    """attn_fwd_tree: q [total,Hq,D] holds the queries of each sequence's last tokens (offsets
    ``cu`` [n + 1]), which form a tree by ``parents`` (None: a chain; one token each: a decoding
    step), over a KVPages ``cache``.

    ``workspace``: a uint8 CUDA tensor, or None to let torch allocate the size that
    attn_fwd_tree_workspace asks for.  Returns (o [total,Hq,D], lse [Hq,total]) without waiting."""
    torch = _torch()
    (total, Hq, D), sq = _rows(q, "q")
    dev = cache.dev
    _same(q, "q", cache.dtype, dev)
    if D != cache.D or Hq % cache.Hkv != 0:
        raise ValueError("q must be [total, Hq, D] with the cache's D and Hq a multiple of its Hkv")
    n = _list(cu, "cu", cache) - 1
    _list(seqs, "seqs", cache, n)
    _list(parents, "parents", cache, total)
    o, lse = _outputs(q, dev, Hq, total, with_lse, out, lse_out, stream)
    so = o.stride()
    if so[2] != 1:
        raise ValueError("out must have its last axis contiguous")
    if workspace is None:
        nbytes = _tree_bytes.get((dev, n, D))
        if nbytes is None:
            with torch.cuda.device(dev):
                st, nbytes = attn_fwd_tree_workspace(n, D)
            if st != ATTN_OK:
                raise AttnError(st, "attn_fwd_tree_workspace")
            _tree_bytes[dev, n, D] = nbytes
        workspace = _new(q, (nbytes,), torch.uint8, stream)
    else:
        nbytes = workspace.numel()
        _same(workspace, "workspace", torch.uint8, dev)
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
    _run("attn_fwd_tree", dev, stream, load().attn_fwd_tree, q.data_ptr(), cache.ref, layer, o.data_ptr(),
         _ptr(lse), cu.data_ptr(), _ptr(seqs), _ptr(parents), n, total, Hq, _Strides4(sq[0], sq[1], so[0], so[1]),
         D ** -0.5 if scale is None else scale, workspace.data_ptr(), nbytes)
    return o, lse
