"""Thin ctypes binding over libgdntree_target.so (include/gdntree_target.h), with the C ABI's names:
the paged key-value cache of the target's attention layers, attention over it, and acceptance at a
temperature.

As in ``_binding``: argument checks, pointer extraction and output allocation only; every step
runs in the library's HIP kernels and there is no fallback.  All tensors of a call lie on the
current device.  Scratch memory is allocated per call unless given, and memory a call allocates
is tied to the stream it runs on.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

from ._binding import Tree, _code, _run

_HERE = os.path.dirname(os.path.abspath(__file__))
TARGET_LIB_PATH = os.path.join(_HERE, "libgdntree_target.so")
GDNTREE_CACHE_BF16, GDNTREE_CACHE_E4M3 = 0, 1
TARGET_EXPORTED = ("gdntree_cache_write", "gdntree_cache_read", "gdntree_cache_commit", "gdntree_attend",
                   "gdntree_attend_workspace", "gdntree_accept_sample", "gdntree_accept_sample_workspace")


class CCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("L", ctypes.c_int), ("pages", ctypes.c_int), ("H_kv", ctypes.c_int),
                ("page_size", ctypes.c_int), ("d", ctypes.c_int), ("dtype", ctypes.c_int)]


def _load() -> ctypes.CDLL:
    from ._binding import CTree
    if not os.path.exists(TARGET_LIB_PATH):
        raise ImportError(f"{TARGET_LIB_PATH} is missing: build it with `python __graft_entry__.py` "
                          "(or __graft_entry__.build())")
    lib = ctypes.CDLL(TARGET_LIB_PATH)
    vp, i, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    for name in ("gdntree_cache_write", "gdntree_cache_read"):
        getattr(lib, name).argtypes = [CCache, i, vp, i, vp, vp, i, i, i, vp, vp, vp]
        getattr(lib, name).restype = i
    lib.gdntree_cache_commit.argtypes = [CCache, vp, i, vp, i, i, i, vp, vp, vp]
    lib.gdntree_cache_commit.restype = i
    lib.gdntree_attend_workspace.argtypes = [i, i, i, i, i]
    lib.gdntree_attend_workspace.restype = sz
    lib.gdntree_attend.argtypes = [CCache, i, vp, i, vp, vp, vp, i, i, i, i, vp, ctypes.c_float, vp, vp, sz, vp]
    lib.gdntree_attend.restype = i
    lib.gdntree_accept_sample_workspace.argtypes = [i, i, i]
    lib.gdntree_accept_sample_workspace.restype = sz
    lib.gdntree_accept_sample.argtypes = [CTree, i, i, i, i, i, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.gdntree_accept_sample.restype = i
    return lib


TARGET_LIB = _load()

_CACHE_CODE = {torch.bfloat16: GDNTREE_CACHE_BF16, torch.float8_e4m3fn: GDNTREE_CACHE_E4M3}


def _arg(t, name: str, dtype, shape, device) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _place(t, name: str, stream):
    """The call's device (that of t, which must be the current one) and stream, and whether the
    stream is another one than the current (memory allocated here is then tied to it)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.device.index != torch.cuda.current_device():
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{torch.cuda.current_device()}")
    current = torch.cuda.current_stream()
    if stream is None:
        return t.device, current.cuda_stream, None
    handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if handle == current.cuda_stream:
        return t.device, handle, None
    return t.device, handle, stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(handle)


def _new(shape, dtype, device, other):
    t = torch.empty(shape, dtype=dtype, device=device)
    if other is not None:
        t.record_stream(other)
    return t


def _scratch(workspace, size: int, device, other):
    if workspace is None:
        workspace = _new(max(size, 16), torch.uint8, device, other)
    elif not isinstance(workspace, torch.Tensor) or workspace.device != device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the call's device")
    return workspace, workspace.numel() * workspace.element_size()


@dataclass
class KVCache:
    """A paged key-value cache of L attention layers: k, v [L][pages][H_kv][page_size][d] (bf16, or
    float8_e4m3fn with the biased exponent bytes of the power-of-two scales in k_scale, v_scale
    uint8 [L][pages][H_kv][page_size]); see gdntree_target.h."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor | None = None
    v_scale: torch.Tensor | None = None

    @staticmethod
    def empty(L: int, pages: int, H_kv: int, page_size: int, d: int, dtype=torch.bfloat16, device="cuda") -> "KVCache":
        if dtype not in _CACHE_CODE:
            raise ValueError(f"unsupported cache dtype {dtype}")
        shape = (L, pages, H_kv, page_size, d)
        k, v = (torch.empty(shape, dtype=dtype, device=device) for _ in range(2))
        if dtype == torch.bfloat16:
            return KVCache(k, v)
        return KVCache(k, v, *(torch.empty(shape[:-1], dtype=torch.uint8, device=device) for _ in range(2)))

    def c(self, device) -> CCache:
        k = self.k
        if k.dtype not in _CACHE_CODE or k.dim() != 5:
            raise ValueError("cache.k must be bf16 or float8_e4m3fn [L][pages][H_kv][page_size][d]")
        code = _CACHE_CODE[k.dtype]
        ks = vs = None
        if code == GDNTREE_CACHE_E4M3:
            if self.k_scale is None or self.v_scale is None:
                raise ValueError("an e4m3 cache needs k_scale and v_scale")
            ks = _arg(self.k_scale, "cache.k_scale", torch.uint8, k.shape[:-1], device)
            vs = _arg(self.v_scale, "cache.v_scale", torch.uint8, k.shape[:-1], device)
        return CCache(_arg(k, "cache.k", k.dtype, k.shape, device), _arg(self.v, "cache.v", k.dtype, k.shape, device),
                      ks, vs, *k.shape, code)


def _table(table, B: int, device):
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        raise ValueError("table must be [B][max_pages]")
    return _arg(table, "table", torch.int32, (B, table.shape[1]), device), table.shape[1]


def gdntree_cache_write(cache: KVCache, layer: int, table, start, k, v, count=None, stream=None,
                        prepare: bool = False) -> None:
    """Rows k, v [B][R][H_kv][d] (bf16 or fp32) into one layer of the cache, row t < count[b] (all R
    when None) of request b at position start[b] + t; see gdntree_target.h."""
    dev, handle, _ = _place(k, "k", stream)
    if k.dim() != 4:
        raise ValueError("k must be [B][R][H_kv][d]")
    B, R, H, D = k.shape
    if cache.k.shape[2] != H or cache.k.shape[4] != D:
        raise ValueError("the rows do not match the cache's heads")
    tp, width = _table(table, B, dev)
    args = (cache.c(dev), int(layer), tp, width, _arg(start, "start", torch.int32, (B,), dev),
            None if count is None else _arg(count, "count", torch.int32, (B,), dev), B, R, _code(k.dtype),
            _arg(k, "k", k.dtype, k.shape, dev), _arg(v, "v", k.dtype, k.shape, dev), handle)
    return _run(TARGET_LIB.gdntree_cache_write, args, prepare, None, (cache, table, start, count, k, v))


def gdntree_cache_read(cache: KVCache, layer: int, table, start, R: int, count=None, out=None,
                       out_dtype=torch.bfloat16, stream=None, prepare: bool = False):
    """Positions start[b] .. start[b] + count[b] - 1 (R of them when count is None) of one layer as
    rows (k, v) [B][R][H_kv][d], in the dtype of `out` or out_dtype; see gdntree_target.h."""
    dev, handle, other = _place(start, "start", stream)
    B, H, D = start.shape[0], cache.k.shape[2], cache.k.shape[4]
    if out is None:
        out = tuple(_new((B, R, H, D), out_dtype, dev, other) for _ in range(2))
    k, v = out
    tp, width = _table(table, B, dev)
    args = (cache.c(dev), int(layer), tp, width, _arg(start, "start", torch.int32, (B,), dev),
            None if count is None else _arg(count, "count", torch.int32, (B,), dev), B, R, _code(k.dtype),
            _arg(k, "k", k.dtype, (B, R, H, D), dev), _arg(v, "v", k.dtype, (B, R, H, D), dev), handle)
    return _run(TARGET_LIB.gdntree_cache_read, args, prepare, (k, v), (cache, table, start, count, k, v))


def gdntree_cache_commit(cache: KVCache, table, ctx_len, acc_len, acc_node, N: int, stream=None,
                         prepare: bool = False) -> None:
    """The accepted path's rows of every layer move together behind the committed positions: position
    ctx_len[b] + acc_node[b][i] to ctx_len[b] + i; see gdntree_target.h."""
    dev, handle, _ = _place(acc_node, "acc_node", stream)
    if acc_node.dim() != 2:
        raise ValueError("acc_node must be [B][P+1]")
    B, P1 = acc_node.shape
    tp, width = _table(table, B, dev)
    args = (cache.c(dev), tp, width, _arg(ctx_len, "ctx_len", torch.int32, (B,), dev), B, int(N), P1 - 1,
            _arg(acc_len, "acc_len", torch.int32, (B,), dev), _arg(acc_node, "acc_node", torch.int32, (B, P1), dev), handle)
    return _run(TARGET_LIB.gdntree_cache_commit, args, prepare, None, (cache, table, ctx_len, acc_len, acc_node))


def gdntree_attend(q, cache: KVCache, layer: int, table, ctx_len, tree: Tree | None = None, n_rows=None,
                   scale: float | None = None, o=None, workspace=None, stream=None, prepare: bool = False):
    """Attention of the new rows q [B][R][H_q][d] (bf16 or fp32) over one layer of the cache, which
    already holds their keys and values at positions ctx_len[b] + t.  With `tree` row t sees its
    ancestors-or-self (tree.anc) and tree.n_nodes rows are in use; without it the rows are a chain,
    n_rows[b] of them (all R when None).  scale: d^-1/2 when None.  Returns o [B][R][H_q][d]; see
    gdntree_target.h."""
    dev, handle, other = _place(q, "q", stream)
    if q.dim() != 4:
        raise ValueError("q must be [B][R][H_q][d]")
    B, R, Hq, D = q.shape
    H = cache.k.shape[2]
    if cache.k.shape[4] != D:
        raise ValueError("q does not match the cache's head size")
    anc = None
    if tree is not None:
        if n_rows is not None:
            raise ValueError("n_rows comes from the tree when one is given")
        anc = _arg(tree.anc, "tree.anc", torch.int64, (B, R), dev)
        n_rows = tree.n_nodes
    tp, width = _table(table, B, dev)
    if o is None:
        o = _new(q.shape, q.dtype, dev, other)
    ws, size = _scratch(workspace, TARGET_LIB.gdntree_attend_workspace(B, R, Hq, H, D), dev, other)
    args = (cache.c(dev), int(layer), tp, width, _arg(ctx_len, "ctx_len", torch.int32, (B,), dev), anc,
            None if n_rows is None else _arg(n_rows, "n_rows", torch.int32, (B,), dev), B, R, Hq, _code(q.dtype),
            _arg(q, "q", q.dtype, q.shape, dev), D ** -0.5 if scale is None else float(scale),
            _arg(o, "o", q.dtype, q.shape, dev), ws.data_ptr(), size, handle)
    return _run(TARGET_LIB.gdntree_attend, args, prepare, o, (q, cache, table, ctx_len, tree, n_rows, o, ws))


def gdntree_accept_sample(tree: Tree, logits, temperature, uniform, P: int, acc=None, workspace=None, stream=None,
                          prepare: bool = False):
    """Acceptance of the tree's drafts against softmax(logits / temperature) from given random numbers,
    and the bonus token: logits [B][N+1][V] (bf16 or fp32), temperature f32 [B] (0: argmax), uniform
    f64 [B][N+1] in [0, 1).  Returns (acc_len [B], acc_tok [B][P+1], acc_node [B][P+1]), as
    gdntree_accept; see gdntree_target.h."""
    dev, handle, other = _place(logits, "logits", stream)
    if logits.dim() != 3:
        raise ValueError("logits must be [B][N+1][V]")
    B, R, V = logits.shape
    if tree.B != B or tree.N != R - 1:
        raise ValueError("tree shape does not match logits")
    if acc is None:
        acc = tuple(_new(s, torch.int32, dev, other) for s in ((B,), (B, P + 1), (B, P + 1)))
    ws, size = _scratch(workspace, TARGET_LIB.gdntree_accept_sample_workspace(B, R - 1, V), dev, other)
    for name in ("parent", "token"):
        _arg(getattr(tree, name), f"tree.{name}", torch.int32, (B, R), dev)
    _arg(tree.n_nodes, "tree.n_nodes", torch.int32, (B,), dev)
    args = (tree.c(), B, R - 1, int(P), V, _code(logits.dtype), _arg(logits, "logits", logits.dtype, logits.shape, dev),
            _arg(temperature, "temperature", torch.float32, (B,), dev),
            _arg(uniform, "uniform", torch.float64, (B, R), dev), _arg(acc[0], "acc_len", torch.int32, (B,), dev),
            _arg(acc[1], "acc_tok", torch.int32, (B, P + 1), dev),
            _arg(acc[2], "acc_node", torch.int32, (B, P + 1), dev), ws.data_ptr(), size, handle)
    return _run(TARGET_LIB.gdntree_accept_sample, args, prepare, tuple(acc),
                (tree, logits, temperature, uniform, acc, ws))
