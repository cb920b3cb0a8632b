"""Thin ctypes binding of the C ABI in ``include/sgqa.h``.

Argument marshalling only: every step of the path runs in ``libsgqa.so``.
Functions take torch tensors (device memory, C-contiguous, in the layouts the
header states) and the current torch CUDA stream.  Errors raise
``SgqaError`` with the library's message.  There is no fallback: if the
library cannot be loaded, importing this module raises.
"""
from __future__ import annotations

import ctypes
import dataclasses
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsgqa.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python -m sparse_long_context_sgqa_b200.build`")
_lib = ctypes.CDLL(LIB_PATH)

STATUS = {0: "SGQA_OK", 1: "SGQA_ERR_INVALID_ARGUMENT", 2: "SGQA_ERR_UNSUPPORTED",
          3: "SGQA_ERR_WORKSPACE", 4: "SGQA_ERR_CUDA", 5: "SGQA_ERR_TIMEOUT", 6: "SGQA_ERR_DEVICE"}

EXPORTED = ["sgqa_workspace_size", "sgqa_merge_blocks", "sgqa_index_topk", "sgqa_sparse_attn",
            "sgqa_sparse_attn_gated", "sgqa_forward", "sgqa_forward_gated", "sgqa_sparse_attn_paged",
            "sgqa_sparse_attn_noalloc",
            "sgqa_workspace_size_q8", "sgqa_kv_append_q8", "sgqa_sparse_attn_q8", "sgqa_forward_q8",
            "sgqa_evict_workspace_size", "sgqa_evict",
            "sgqa_set_wait_limit_ns", "sgqa_check", "sgqa_last_error", "sgqa_version", "sgqa_launch_count"]


class SgqaError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__(f"{STATUS.get(code, code)}: {msg}")
        self.code = code


class _Params(ctypes.Structure):
    _fields_ = [("num_kv_groups", ctypes.c_int32), ("heads_per_group", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("idx_heads", ctypes.c_int32),
                ("idx_dim", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("topk", ctypes.c_int32), ("merge_in_f32", ctypes.c_int32),
                ("scale", ctypes.c_float)]


class _CacheArray(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("block_bytes", ctypes.c_int64), ("tail_only", ctypes.c_int32)]


@dataclasses.dataclass
class Params:
    __slots__ = ("_struct", "__dict__", "__weakref__")  # the C structure stays out of the fields' dictionary

    num_kv_groups: int = 4
    heads_per_group: int = 16
    head_dim: int = 192
    idx_heads: int = 8
    idx_dim: int = 64
    block_size: int = 8
    topk: int = 512
    merge_in_f32: int = 0
    scale: float = 0.0

    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        object.__setattr__(self, "_struct", None)  # built again by the next call

    def c(self) -> _Params:
        c = getattr(self, "_struct", None)
        if c is None:
            c = _Params(self.num_kv_groups, self.heads_per_group, self.head_dim, self.idx_heads, self.idx_dim,
                        self.block_size, self.topk, self.merge_in_f32, self.scale)
            object.__setattr__(self, "_struct", c)
        return c

    def __getstate__(self):
        return dict(self.__dict__)

    def __setstate__(self, state):
        self.__dict__.update(state)


_vp, _i64, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
_P = ctypes.POINTER(_Params)
_lib.sgqa_workspace_size.argtypes = [_P, _i64, _i64, _i64, ctypes.POINTER(_sz)]
_lib.sgqa_merge_blocks.argtypes = [_P, _i64, _i64, _vp, _vp, _i64, _i64, _vp, _vp, _vp]
_lib.sgqa_index_topk.argtypes = [_P, _i64, _i64, _i64, _vp, _vp, _i64, _vp, _vp, _vp, _vp, _sz, _vp]
_lib.sgqa_sparse_attn.argtypes = [_P, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _vp, _vp, _vp,
                                  _vp, _sz, _vp]
_lib.sgqa_sparse_attn_gated.argtypes = [_P, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp,
                                        _vp, _sz, _vp]
_lib.sgqa_forward.argtypes = [_P, _i64, _i64, _i64, _vp, _vp, _vp, _i64, _i64, _vp, _vp, _vp, _vp,
                              _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
_lib.sgqa_forward_gated.argtypes = [_P, _i64, _i64, _i64, _vp, _vp, _vp, _i64, _i64, _vp, _vp, _vp, _vp,
                                    _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
_lib.sgqa_sparse_attn_paged.argtypes = [_P, _i64, _i64, _i64, _vp, _vp, _vp, _i64, _vp, _i64, _i64, _vp, _vp, _vp,
                                        _vp, _vp, _sz, _vp]
_lib.sgqa_sparse_attn_noalloc.argtypes = [_P, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp]
_lib.sgqa_workspace_size_q8.argtypes = [_P, _i64, _i64, _i64, ctypes.POINTER(_sz)]
_lib.sgqa_kv_append_q8.argtypes = [_P, _i64, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp]
_lib.sgqa_sparse_attn_q8.argtypes = [_P, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                     _sz, _vp]
_lib.sgqa_forward_q8.argtypes = [_P, _i64, _i64, _i64, _vp, _vp, _vp, _i64] + [_vp] * 15 + [_sz, _vp]
_lib.sgqa_evict_workspace_size.argtypes = [_P, _i64, _i64, ctypes.POINTER(_sz)]
_lib.sgqa_evict.argtypes = [_P, _i64, _i64, _i64, _i64, _i64, _i64, _vp, _vp, _i64, _i64, _vp, _vp,
                            ctypes.POINTER(_CacheArray), ctypes.c_int32, _vp, _sz, _vp]
_lib.sgqa_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
_lib.sgqa_check.argtypes = [_vp]
_lib.sgqa_last_error.restype = ctypes.c_char_p
_lib.sgqa_version.restype = ctypes.c_char_p
_lib.sgqa_launch_count.restype = ctypes.c_uint64
for _f in EXPORTED[:-3]:
    getattr(_lib, _f).restype = ctypes.c_int


def _ok(code):
    if code != 0:
        raise SgqaError(code, _lib.sgqa_last_error().decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def version() -> str:
    return _lib.sgqa_version().decode()


def launch_count() -> int:
    """Kernels launched by the library so far in this process."""
    return int(_lib.sgqa_launch_count())


def sgqa_workspace_size(p: Params, num_seqs: int, nq: int, max_ctx: int) -> int:
    out = _sz(0)
    _ok(_lib.sgqa_workspace_size(ctypes.byref(p.c()), num_seqs, nq, max_ctx, ctypes.byref(out)))
    return out.value


def alloc_workspace(p: Params, num_seqs: int, nq: int, max_ctx: int, device) -> torch.Tensor:
    n = sgqa_workspace_size(p, num_seqs, nq, max_ctx)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def sgqa_merge_blocks(p: Params, num_seqs, cache_cap, proxy_k, comp_logits, blk_begin, blk_end,
                      merged_f32, store, stream=None):
    _ok(_lib.sgqa_merge_blocks(ctypes.byref(p.c()), num_seqs, cache_cap, _ptr(proxy_k), _ptr(comp_logits),
                               blk_begin, blk_end, _ptr(merged_f32), _ptr(store), _stream(stream)))


def sgqa_index_topk(p: Params, num_seqs, q_pos0, nq, idx_q, idx_w, cache_cap, store, sel, sel_count,
                    workspace, stream=None):
    _ok(_lib.sgqa_index_topk(ctypes.byref(p.c()), num_seqs, q_pos0, nq, _ptr(idx_q), _ptr(idx_w), cache_cap,
                             _ptr(store), _ptr(sel), _ptr(sel_count), _ptr(workspace),
                             workspace.numel() if workspace is not None else 0, _stream(stream)))


def sgqa_sparse_attn(p: Params, num_seqs, q_pos0, nq, q, cache_cap, cache_len, k_cache, v_cache, sel,
                     sel_count, out, workspace, stream=None):
    _ok(_lib.sgqa_sparse_attn(ctypes.byref(p.c()), num_seqs, q_pos0, nq, _ptr(q), cache_cap, cache_len,
                              _ptr(k_cache), _ptr(v_cache), _ptr(sel), _ptr(sel_count), _ptr(out),
                              _ptr(workspace), workspace.numel() if workspace is not None else 0,
                              _stream(stream)))


def sgqa_sparse_attn_gated(p: Params, num_seqs, q_pos0, nq, q, cache_cap, cache_len, k_cache, v_cache, sel,
                           sel_count, gate, out, workspace, stream=None):
    """sgqa_sparse_attn with the head-wise sigmoid output gate (gate: [S, nq, G*Hg] bf16 logits)."""
    _ok(_lib.sgqa_sparse_attn_gated(ctypes.byref(p.c()), num_seqs, q_pos0, nq, _ptr(q), cache_cap, cache_len,
                                    _ptr(k_cache), _ptr(v_cache), _ptr(sel), _ptr(sel_count), _ptr(gate),
                                    _ptr(out), _ptr(workspace), workspace.numel() if workspace is not None else 0,
                                    _stream(stream)))


def sgqa_forward_gated(p: Params, num_seqs, q_pos0, nq, q, idx_q, idx_w, cache_cap, cache_len, proxy_k,
                       comp_logits, k_cache, v_cache, merged_f32, store, sel, sel_count, gate, out, workspace,
                       stream=None):
    """sgqa_forward with the head-wise sigmoid output gate (gate: [S, nq, G*Hg] bf16 logits)."""
    _ok(_lib.sgqa_forward_gated(ctypes.byref(p.c()), num_seqs, q_pos0, nq, _ptr(q), _ptr(idx_q), _ptr(idx_w),
                                cache_cap, cache_len, _ptr(proxy_k), _ptr(comp_logits), _ptr(k_cache),
                                _ptr(v_cache), _ptr(merged_f32), _ptr(store), _ptr(sel), _ptr(sel_count),
                                _ptr(gate), _ptr(out), _ptr(workspace),
                                workspace.numel() if workspace is not None else 0, _stream(stream)))


def sgqa_forward(p: Params, num_seqs, q_pos0, nq, q, idx_q, idx_w, cache_cap, cache_len, proxy_k,
                 comp_logits, k_cache, v_cache, merged_f32, store, sel, sel_count, out, workspace,
                 stream=None):
    _ok(_lib.sgqa_forward(ctypes.byref(p.c()), num_seqs, q_pos0, nq, _ptr(q), _ptr(idx_q), _ptr(idx_w),
                          cache_cap, cache_len, _ptr(proxy_k), _ptr(comp_logits), _ptr(k_cache),
                          _ptr(v_cache), _ptr(merged_f32), _ptr(store), _ptr(sel), _ptr(sel_count),
                          _ptr(out), _ptr(workspace), workspace.numel() if workspace is not None else 0,
                          _stream(stream)))


def sgqa_sparse_attn_paged(p: Params, num_seqs, q_pos0, nq, q, k_pool, v_pool, page_table, cache_len, sel,
                           sel_count, out, gate=None, workspace=None, stream=None):
    """Attention over a paged cache: pools [num_pages, G, 16, D], page_table [S, max_pages] int32;
    a workspace only for calls of more than 32 queries per sequence."""
    num_pages = k_pool.shape[0]
    _ok(_lib.sgqa_sparse_attn_paged(ctypes.byref(p.c()), num_seqs, q_pos0, nq, _ptr(q), _ptr(k_pool), _ptr(v_pool),
                                    num_pages, _ptr(page_table), page_table.shape[1], cache_len, _ptr(sel),
                                    _ptr(sel_count), _ptr(gate), _ptr(out), _ptr(workspace),
                                    workspace.numel() if workspace is not None else 0, _stream(stream)))


def sgqa_sparse_attn_noalloc(p: Params, num_seqs, q_pos0, nq, q, cache_cap, cache_len, k_cache, v_cache, sel,
                             sel_count, out, stream=None):
    """sgqa_sparse_attn for decode-sized calls (nq <= 32) using the library's
    static scratch instead of a workspace; for callers that cannot allocate."""
    _ok(_lib.sgqa_sparse_attn_noalloc(ctypes.byref(p.c()), num_seqs, q_pos0, nq, _ptr(q), cache_cap, cache_len,
                                      _ptr(k_cache), _ptr(v_cache), _ptr(sel), _ptr(sel_count), _ptr(out),
                                      _stream(stream)))


def sgqa_workspace_size_q8(p: Params, num_seqs: int, nq: int, max_ctx: int) -> int:
    out = _sz(0)
    _ok(_lib.sgqa_workspace_size_q8(ctypes.byref(p.c()), num_seqs, nq, max_ctx, ctypes.byref(out)))
    return out.value


def alloc_workspace_q8(p: Params, num_seqs: int, nq: int, max_ctx: int, device) -> torch.Tensor:
    n = sgqa_workspace_size_q8(p, num_seqs, nq, max_ctx)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def _check(name, t, dtype, numel, dev):
    """Address of a contiguous tensor of the values the call reads or writes there, on CUDA device `dev`."""
    if t.dtype is dtype and t.numel() == numel and t.is_cuda and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{name}: expected a contiguous CUDA tensor of {numel} {dtype} values on the other tensors' device, "
                     f"got {tuple(t.shape)} {t.dtype} on {t.device}{'' if t.is_contiguous() else ', not contiguous'}")


# the current stream's handle without an object around it, where torch has that (a few microseconds per call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _run(fn, lead, stream, *args):
    """Call fn on the tensors' own device, on the given stream or that device's current one."""
    index = lead.get_device()
    if stream is None:
        raw = _raw_stream(index)
    elif stream.device.index == index:
        raw = stream.cuda_stream
    else:
        raise ValueError(f"the stream belongs to {stream.device}, the tensors to {lead.device}")
    if index == torch.cuda.current_device():
        _ok(fn(*args, raw))
    else:
        with torch.cuda.device(index):
            _ok(fn(*args, raw))


def _q8_cache(p, S, cap, kv8, kv_scale, dev):
    n = S * cap // 8 * p.num_kv_groups * 2
    return _check("kv8", kv8, torch.uint8, n * 8 * p.head_dim, dev), _check("kv_scale", kv_scale, torch.float32, n, dev)


def _workspace(ws, dev):
    if ws is None:
        return None, 0
    n = ws.numel()
    return _check("workspace", ws, torch.uint8, n, dev), n


def sgqa_kv_append_q8(p: Params, num_seqs, cache_cap, pos0, n, k, v, tail, kv8, kv_scale, stream=None):
    """Quantise the K/V rows of positions [pos0, pos0 + n) (k, v: [S, n, G, D] bf16) into the 8-bit cache."""
    row, dev = num_seqs * p.num_kv_groups * p.head_dim, kv8.get_device()
    _run(_lib.sgqa_kv_append_q8, kv8, stream, ctypes.byref(p.c()), num_seqs, cache_cap, pos0, n,
         _check("k", k, torch.bfloat16, row * n, dev), _check("v", v, torch.bfloat16, row * n, dev),
         None if tail is None else _check("tail", tail, torch.bfloat16, row * 16, dev),
         *_q8_cache(p, num_seqs, cache_cap, kv8, kv_scale, dev))


def sgqa_sparse_attn_q8(p: Params, num_seqs, q_pos0, nq, q, cache_cap, cache_len, kv8, kv_scale, sel, sel_count, out,
                        workspace=None, gate=None, acc=None, stream=None):
    """Attention over the 8-bit cache; acc ([S, cache_cap / 8] int64, units of 2^-32) gains the blocks' weights."""
    rows = num_seqs * nq * p.num_kv_groups
    heads, dev = rows * p.heads_per_group, kv8.get_device()
    _run(_lib.sgqa_sparse_attn_q8, kv8, stream, ctypes.byref(p.c()), num_seqs, q_pos0, nq,
         _check("q", q, torch.bfloat16, heads * p.head_dim, dev), cache_cap, cache_len,
         *_q8_cache(p, num_seqs, cache_cap, kv8, kv_scale, dev), _check("sel", sel, torch.int32, rows * p.topk, dev),
         _check("sel_count", sel_count, torch.int32, rows, dev),
         None if gate is None else _check("gate", gate, torch.bfloat16, heads, dev),
         None if acc is None else _check("acc", acc, torch.int64, num_seqs * cache_cap // 8, dev),
         _check("out", out, torch.bfloat16, heads * p.head_dim, dev), *_workspace(workspace, dev))


def sgqa_forward_q8(p: Params, num_seqs, q_pos0, nq, q, idx_q, idx_w, cache_cap, proxy_k, comp_logits, k, v, tail, kv8,
                    kv_scale, merged_f32, store, sel, sel_count, out, workspace, gate=None, acc=None, stream=None):
    """merge -> append (k, v: the call's own rows) -> index/top-k -> attention over the 8-bit cache."""
    rows = num_seqs * nq * p.num_kv_groups
    heads, blocks = rows * p.heads_per_group, num_seqs * cache_cap // 8
    in_dt = torch.float32 if p.merge_in_f32 else torch.bfloat16
    dev = kv8.get_device()
    kv, sc = _q8_cache(p, num_seqs, cache_cap, kv8, kv_scale, dev)
    _run(_lib.sgqa_forward_q8, kv8, stream, ctypes.byref(p.c()), num_seqs, q_pos0, nq,
         _check("q", q, torch.bfloat16, heads * p.head_dim, dev),
         _check("idx_q", idx_q, torch.bfloat16, rows * p.idx_heads * p.idx_dim, dev),
         _check("idx_w", idx_w, torch.float32, rows * p.idx_heads, dev), cache_cap,
         _check("proxy_k", proxy_k, in_dt, num_seqs * cache_cap * p.idx_dim, dev),
         _check("comp_logits", comp_logits, in_dt, num_seqs * cache_cap * p.idx_dim, dev),
         _check("k", k, torch.bfloat16, rows * p.head_dim, dev), _check("v", v, torch.bfloat16, rows * p.head_dim, dev),
         None if tail is None else _check("tail", tail, torch.bfloat16, num_seqs * 16 * p.num_kv_groups * p.head_dim, dev),
         kv, sc, None if merged_f32 is None else _check("merged_f32", merged_f32, torch.float32, blocks * p.idx_dim, dev),
         _check("store", store, torch.uint8, blocks * p.idx_dim, dev), _check("sel", sel, torch.int32, rows * p.topk, dev),
         _check("sel_count", sel_count, torch.int32, rows, dev),
         None if gate is None else _check("gate", gate, torch.bfloat16, heads, dev),
         None if acc is None else _check("acc", acc, torch.int64, blocks, dev),
         _check("out", out, torch.bfloat16, heads * p.head_dim, dev), *_workspace(workspace, dev))


def sgqa_evict_workspace_size(p: Params, num_seqs: int, cache_cap: int) -> int:
    out = _sz(0)
    _ok(_lib.sgqa_evict_workspace_size(ctypes.byref(p.c()), num_seqs, cache_cap, ctypes.byref(out)))
    return out.value


def alloc_evict_workspace(p: Params, num_seqs: int, cache_cap: int, device) -> torch.Tensor:
    return torch.empty(max(sgqa_evict_workspace_size(p, num_seqs, cache_cap), 256), dtype=torch.uint8, device=device)


def sgqa_evict(p: Params, num_seqs, cache_cap, cache_len, keep, first, recent, acc, pos, pos_count, evicted, acc_out,
               pos_out, arrays, workspace, tail_arrays=(), stream=None):
    """Keep the `keep` heaviest blocks of every sequence.  arrays: contiguous tensors whose leading dimensions are
    (sequence, block) or (sequence, token); tail_arrays: the same, of which only the incomplete block moves."""
    blocks = num_seqs * (cache_cap // p.block_size)
    n, dev = len(arrays) + len(tail_arrays), acc.get_device()
    c = (_CacheArray * max(1, n))()
    for i, t in enumerate((*arrays, *tail_arrays) if tail_arrays else arrays):
        size = t.nbytes
        if not t.is_cuda or t.get_device() != dev or not t.is_contiguous() or blocks == 0 or size % blocks:
            raise ValueError("evict: every array is a contiguous tensor of cache_cap / block_size blocks per sequence on acc's "
                             "CUDA device")
        c[i] = (t.data_ptr(), size // blocks, i >= len(arrays))
    _run(_lib.sgqa_evict, acc, stream, ctypes.byref(p.c()), num_seqs, cache_cap, cache_len, keep, first, recent,
         _check("acc", acc, torch.int64, blocks, dev), None if pos is None else _check("pos", pos, torch.int32, blocks, dev),
         pos_count, evicted, _check("acc_out", acc_out, torch.int64, blocks, dev), _check("pos_out", pos_out, torch.int32, blocks, dev),
         c, n, *_workspace(workspace, dev))


def sgqa_set_wait_limit_ns(ns: int):
    """Time limit of the kernels' pipeline waits on the current device (0: the default, 2 s)."""
    _ok(_lib.sgqa_set_wait_limit_ns(int(ns)))


def sgqa_check(stream=None):
    _ok(_lib.sgqa_check(_stream(stream)))
