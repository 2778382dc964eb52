"""Python binding of libkascade (include/kascade.h).

Argument marshalling only: every step of the attention path runs in the
library's CUDA kernels. PyTorch supplies device memory (outputs, the
workspace) and the current CUDA stream. Importing this module loads
``libkascade.so`` from this package directory and raises if it is missing;
there is no fallback.
"""
import contextlib
import ctypes
import functools
import math
import os
from typing import List, Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkascade.so")

if not os.path.exists(LIB_PATH):
    raise ImportError("libkascade.so is not built; run python -m long_context_anchor_gb300.build "
                      "(or __graft_entry__.build())")
_lib = ctypes.CDLL(LIB_PATH)

OK, INVALID_ARG, UNSUPPORTED, WORKSPACE, CUDA, BAD_INPUT, TIMEOUT = range(7)
F32, BF16 = 0, 1
DECODE, PREFILL = 0, 1
PER_QHEAD, PER_KVHEAD = 0, 1     # kascade_index_mode: per query head, or GQA-pooled
TILE = 128


class Desc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("n_q_heads", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("kv_len", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("scale", ctypes.c_float), ("group_map", ctypes.POINTER(ctypes.c_int32)),
                ("index_mode", ctypes.c_int32)]


class QCache(ctypes.Structure):
    """kascade_qcache: geometry of a paged 4-bit key/value cache."""
    _fields_ = [("block_size", ctypes.c_int32), ("num_blocks", ctypes.c_int32),
                ("max_blocks", ctypes.c_int32), ("k_scale", ctypes.c_float),
                ("v_scale", ctypes.c_float)]


class QCacheStep(ctypes.Structure):
    """kascade_qcache_step: the device state one decode step works on."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("block_table", "kv_lens", "new_lens", "free_blocks",
                                               "free_count", "cu_new", "slot_map")]
    _fields_ += [("max_new", ctypes.c_int32)]


_vp, _i32, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
_DP = ctypes.POINTER(Desc)
_QP, _I64P = ctypes.POINTER(QCache), ctypes.POINTER(ctypes.c_int64)
_SIGS = {
    "kascade_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "kascade_workspace_size": (_sz, [_DP, _i32, _i32]),
    "kascade_workspace_init": (ctypes.c_int, [_vp, _sz, _vp]),
    "kascade_device_error": (ctypes.c_int, [_vp, _vp]),
    "kascade_check_wait_timeout": (ctypes.c_int, [_vp, _sz, _vp]),
    "kascade_dense_decode": (ctypes.c_int, [_DP, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "kascade_anchor_decode": (ctypes.c_int, [_DP, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _sz, _vp]),
    "kascade_anchor_decode_fused": (ctypes.c_int, [_DP, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _vp,
                                                   _sz, _vp]),
    "kascade_reuse_decode": (ctypes.c_int, [_DP, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _sz, _vp]),
    "kascade_topk": (ctypes.c_int, [_vp, _i32, _i32, _i32, _vp, _vp, _sz, _vp]),
    "kascade_dense_decode_noalloc": (ctypes.c_int, [_DP, _vp, _vp, _vp, _vp, _vp]),
    "kascade_noalloc_device_error": (ctypes.c_int, [_vp]),
    "kascade_anchor_decode_shard": (ctypes.c_int, [_DP, _vp, _vp, _vp, _i32, _i32, _vp, _vp, _vp,
                                                   _vp, _vp, _sz, _vp]),
    "kascade_merge_workspace_size": (_sz, [_DP, _i32, _i32]),
    "kascade_merge_decode_shards": (ctypes.c_int, [_DP, _i32, _vp, _vp, _vp, _vp, _i32, _vp, _vp,
                                                   _vp, _sz, _vp]),
    "kascade_dense_prefill": (ctypes.c_int, [_DP, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "kascade_anchor_prefill": (ctypes.c_int, [_DP, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _sz,
                                              _vp]),
    "kascade_reuse_prefill": (ctypes.c_int, [_DP, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _sz, _vp]),
    "kascade_run_stack": (ctypes.c_int, [_DP, _i32, _i32, ctypes.POINTER(_vp), ctypes.POINTER(_vp),
                                         ctypes.POINTER(_vp), _i32, ctypes.POINTER(_i32), _i32,
                                         ctypes.POINTER(_vp), _vp, _vp, _sz, _vp]),
    "kascade_run_stack_profiled": (ctypes.c_int, [_DP, _i32, _i32, ctypes.POINTER(_vp),
                                                  ctypes.POINTER(_vp), ctypes.POINTER(_vp), _i32,
                                                  ctypes.POINTER(_i32), _i32, ctypes.POINTER(_vp),
                                                  _vp, _vp, _sz, _vp, ctypes.POINTER(_vp)]),
    "kascade_qcache_bytes": (_sz, [_QP, _i32, _i32]),
    "kascade_qcache_workspace_size": (_sz, [_DP, _QP, _i32]),
    "kascade_qcache_reuse_workspace_size": (_sz, [_DP, _QP, _i32]),
    "kascade_qcache_plan": (ctypes.c_int, [_QP, _i32] + [_vp] * 9 + [_i32, _vp, _sz, _vp]),
    "kascade_qcache_append": (ctypes.c_int, [_QP, _i32, _i32, _i32, _vp, _vp, _I64P, _vp, _i32,
                                             _vp, _vp, _sz, _vp]),
    "kascade_qcache_read": (ctypes.c_int, [_QP, _i32, _i32, _i32, _vp, _vp, _i32, _vp, _vp, _I64P,
                                           _vp, _sz, _vp]),
    "kascade_qcache_dense_decode": (ctypes.c_int, [_DP, _QP] + [_vp] * 7 + [_sz, _vp]),
    "kascade_qcache_anchor_decode": (ctypes.c_int, [_DP, _QP] + [_vp] * 4 + [_i32] + [_vp] * 4 +
                                     [_sz, _vp]),
    "kascade_qcache_reuse_decode": (ctypes.c_int, [_DP, _QP] + [_vp] * 4 + [_i32] + [_vp] * 3 +
                                    [_sz, _vp]),
    "kascade_qcache_run_stack": (ctypes.c_int, [_DP, _QP, ctypes.POINTER(QCacheStep), _i32] +
                                 [ctypes.POINTER(_vp)] * 4 +
                                 [_i32, ctypes.POINTER(_i32), _i32, ctypes.POINTER(_vp), _vp, _vp,
                                  _sz, _vp]),
    "kascade_overlap_workspace_size": (_sz, [_i32, _i32, _i32]),
    "kascade_calibrate_workspace_size": (_sz, [_DP, _i32, _i32]),
    "kascade_calibrate": (ctypes.c_int, [_DP, _i32, ctypes.POINTER(_vp), ctypes.POINTER(_vp),
                                         ctypes.POINTER(_vp), _i32, ctypes.POINTER(_vp), _vp,
                                         ctypes.POINTER(ctypes.c_double), _vp, _sz, _vp]),
    "kascade_calibrate_recall_workspace_size": (_sz, [_DP, _i32, _i32]),
    "kascade_calibrate_recall": (ctypes.c_int, [_DP, _i32, ctypes.POINTER(_vp), ctypes.POINTER(_vp),
                                                ctypes.POINTER(_vp), _i32, ctypes.POINTER(_vp), _vp,
                                                ctypes.POINTER(ctypes.c_double), _vp, _sz, _vp]),
    "kascade_layer_overlap": (ctypes.c_int, [_vp, _i32, _i32, _i32, _i32, _vp, _vp, _sz, _vp]),
    "kascade_schedule_anchors": (ctypes.c_int, [ctypes.POINTER(ctypes.c_double), _i32, _i32,
                                                ctypes.POINTER(_i32), ctypes.POINTER(ctypes.c_double)]),
}
for _name, (_res, _args) in _SIGS.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args

EXPORTED = tuple(_SIGS)


class KascadeError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__("%s: %s (status %d)" % (where, status_string(status), status))
        self.status = status


def status_string(s: int) -> str:
    return _lib.kascade_status_string(int(s)).decode()


def _check(status: int, where: str):
    if status != OK:
        raise KascadeError(status, where)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def make_desc(batch, n_q_heads, n_kv_heads, head_dim, kv_len, dtype, scale=0.0,
              group_map: Optional[Sequence[int]] = None, pooled: bool = False):
    d = Desc(batch, n_q_heads, n_kv_heads, head_dim, kv_len, dtype,
             float(scale or 0.0), None, PER_KVHEAD if pooled else PER_QHEAD)
    keep = None
    if group_map is not None:
        keep = (ctypes.c_int32 * n_q_heads)(*[int(x) for x in group_map])
        d.group_map = ctypes.cast(keep, ctypes.POINTER(ctypes.c_int32))
    d._keep = keep      # keep the host array alive with the descriptor
    return d


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError("q/k/v must be bfloat16 or float32")


def decode_desc(q, k, group_map=None, scale=None, pooled=False):
    B, Hq, d = q.shape
    _, Hkv, N, _ = k.shape
    return make_desc(B, Hq, Hkv, d, N, _dtype_code(q), scale or 0.0, group_map, pooled)


def prefill_desc(q, k, group_map=None, scale=None, pooled=False):
    B, Hq, N, d = q.shape
    Hkv = k.shape[1]
    return make_desc(B, Hq, Hkv, d, N, _dtype_code(q), scale or 0.0, group_map, pooled)


def workspace_size(desc, topk: int, mode: int) -> int:
    n = _lib.kascade_workspace_size(ctypes.byref(desc), int(topk), int(mode))
    if n == 0:
        raise KascadeError(INVALID_ARG, "kascade_workspace_size")
    return n


class Workspace:
    """Caller-owned device workspace (torch memory), zeroed once when (re)allocated."""

    def __init__(self, device=None):
        self.device = torch.device(device if device is not None else "cuda")
        self.buf: Optional[torch.Tensor] = None
        self.captured = False     # a graph holds the buffer's address

    def get(self, nbytes: int, stream=None) -> torch.Tensor:
        old = self.buf
        if old is None or old.numel() < nbytes:
            if self.captured:
                raise RuntimeError("this workspace was captured into a CUDA graph, which holds its "
                                   "address: it cannot grow to %d bytes (use another one, or size "
                                   "it before the capture)" % nbytes)
            self.buf = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=self.device)
            _check(_lib.kascade_workspace_init(_ptr(self.buf), self.buf.numel(), _stream(stream)),
                   "kascade_workspace_init")
            if old is not None and not (old.is_cuda and torch.cuda.is_current_stream_capturing()):
                self._carry(old, stream)
        return self.buf

    def _carry(self, old, stream):
        """A device error that waits to be read in the smaller buffer goes into the new
        one; the old one's memory is kept until the stream, which may be another than
        its own, has done with it."""
        if not old.is_cuda:
            self.buf[:8].copy_(old[:8])
            return
        s = stream if stream is not None else torch.cuda.current_stream(old.device)
        old.record_stream(s)
        with torch.cuda.stream(s):
            self.buf[:8].copy_(old[:8])

    def check_wait_timeout(self, stream=None) -> int:
        """Run one device wait that can only time out; returns the device error status."""
        buf = self.get(256, stream)
        _check(_lib.kascade_check_wait_timeout(_ptr(buf), buf.numel(), _stream(stream)),
               "kascade_check_wait_timeout")
        return self.device_error(stream)

    def device_error(self, stream=None) -> int:
        """Synchronise and read/clear the device error word (an int status)."""
        if self.buf is None:
            return OK
        return _lib.kascade_device_error(_ptr(self.buf), _stream(stream))


_default_ws = {}


def default_workspace(device, stream=None) -> Workspace:
    """The workspace of calls that name none: one per device, and one more per
    stream other than the device's default one for the cache calls (qcache_*),
    so that those on two streams do not share one. Threads that call on one stream
    at a time need a workspace each. stream: torch.cuda.Stream."""
    dev = torch.device(device)
    index = dev.index if dev.index is not None else torch.cuda.current_device()
    raw = 0 if stream is None else stream.cuda_stream
    return _workspace_of(index, raw)


def _workspace_of(index, raw):
    key = (index, raw) if raw else index
    if key not in _default_ws:
        _default_ws[key] = Workspace(torch.device("cuda", index))
    return _default_ws[key]


def _ws(ws, device, nbytes, stream):
    ws = ws if ws is not None else default_workspace(device)
    buf = ws.get(nbytes, stream)
    return ws, buf


# The library reads and writes raw device pointers with the extents the
# descriptor implies, so every tensor is checked against those extents here,
# before its address is handed over: a wrong shape, dtype or device would
# otherwise become an out-of-bounds access on the GPU.

def _expect(t, name, shape, dtype):
    """Shape, dtype and contiguity of one tensor (no device check)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s: expected a torch.Tensor" % name)
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s: shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if t.dtype != dtype:
        raise TypeError("%s: dtype %s, expected %s" % (name, t.dtype, dtype))
    if not t.is_contiguous():
        raise ValueError("%s: must be contiguous" % name)


_DEVICE_TYPE = "cuda"   # the only device type whose addresses the library takes


def _same_cuda_device(named):
    """All tensors on one CUDA device; returns it."""
    dev = named[0][1].device
    if dev.type != _DEVICE_TYPE:
        raise ValueError("%s: on %s; the library takes CUDA device tensors" % (named[0][0], dev))
    for name, t in named[1:]:
        if t.device != dev:
            raise ValueError("%s: on %s, expected %s" % (name, t.device, dev))
    return dev


def _attn_inputs(q, k, v, prefill: bool):
    """Validated (B, Hq, Hkv, N, d) of one layer's q, k, v.

    decode: q [B,Hq,d], k/v [B,Hkv,N,d]; prefill: q [B,Hq,N,d], k/v [B,Hkv,N,d].
    k and v take q's dtype (bf16 or fp32)."""
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor):
            raise TypeError("%s: expected a torch.Tensor" % name)
    if q.dim() != (4 if prefill else 3) or k.dim() != 4:
        raise ValueError("q must be %s and k, v [B,Hkv,N,d]; got q %s, k %s"
                         % ("[B,Hq,N,d]" if prefill else "[B,Hq,d]", tuple(q.shape),
                            tuple(k.shape)))
    _dtype_code(q)
    B, Hq, d = q.shape[0], q.shape[1], q.shape[-1]
    Hkv, N = k.shape[1], k.shape[2]
    if prefill and q.shape[2] != N:
        raise ValueError("q: %d rows, k: %d keys; prefill needs both equal" % (q.shape[2], N))
    _expect(q, "q", q.shape, q.dtype)
    _expect(k, "k", (B, Hkv, N, d), q.dtype)
    _expect(v, "v", (B, Hkv, N, d), q.dtype)
    return B, Hq, Hkv, N, d


def _all_like(ts, name, shape, dtype, dev):
    """Every tensor of a per-layer list has this shape, dtype and device and is
    contiguous (one fast pass; the first mismatch gets a detailed error)."""
    for l, t in enumerate(ts):
        if not (isinstance(t, torch.Tensor) and t.shape == shape and t.dtype == dtype
                and t.device == dev and t.is_contiguous()):
            _expect(t, "%s[%d]" % (name, l), shape, dtype)
            raise ValueError("%s[%d]: on %s, expected %s" % (name, l, t.device, dev))


def _layers(qs, ks, vs, prefill: bool):
    """Validated stack inputs: every layer has layer 0's shapes, dtype and
    device; returns (B, Hq, Hkv, N, d) and the device."""
    L = len(qs)
    if L < 1 or len(ks) != L or len(vs) != L:
        raise ValueError("qs, ks, vs: one tensor per layer each (got %d, %d, %d)"
                         % (len(qs), len(ks), len(vs)))
    sizes = _attn_inputs(qs[0], ks[0], vs[0], prefill)
    dev = _same_cuda_device([("qs[0]", qs[0]), ("ks[0]", ks[0]), ("vs[0]", vs[0])])
    _all_like(qs, "qs", qs[0].shape, qs[0].dtype, dev)
    _all_like(ks, "ks", ks[0].shape, qs[0].dtype, dev)
    _all_like(vs, "vs", ks[0].shape, qs[0].dtype, dev)
    return sizes, dev


# ------------------------------------------------------------------ decode --

def dense_decode(q, k, v, group_map=None, scale=None, out=None, ws=None, stream=None):
    """Exact decode attention: q [B,Hq,d], k/v [B,Hkv,N,d] -> out [B,Hq,d]."""
    _attn_inputs(q, k, v, prefill=False)
    if out is not None:
        _expect(out, "out", q.shape, q.dtype)
    _same_cuda_device([("q", q), ("k", k), ("v", v)] + ([("out", out)] if out is not None else []))
    desc = decode_desc(q, k, group_map, scale)
    out = torch.empty_like(q) if out is None else out
    ws, buf = _ws(ws, q.device, workspace_size(desc, 1, DECODE), stream)
    _check(_lib.kascade_dense_decode(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(out),
                                     _ptr(buf), buf.numel(), _stream(stream)), "kascade_dense_decode")
    return out


def anchor_decode(q, k, v, topk, group_map=None, scale=None, return_scores=False, out=None,
                  idx=None, ws=None, stream=None, pooled=False, fused=False):
    """Anchor layer: (out [B,Hq,d], idx [B,H,topk] int32[, scores [B,H,N] fp32]).

    H = Hq: per-head sets, scores = the scaled logits. pooled: H = Hkv, one
    set per KV head, scores = the group sums of the softmax weights. fused:
    the Top-k fused into the attention kernel (kascade_anchor_decode_fused;
    bf16, per-head sets; the same results)."""
    B, Hq, Hkv, N, _ = _attn_inputs(q, k, v, prefill=False)
    H = Hkv if pooled else Hq
    extra = []
    if out is not None:
        _expect(out, "out", q.shape, q.dtype)
        extra.append(("out", out))
    if idx is not None:
        _expect(idx, "idx", (B, H, topk), torch.int32)
        extra.append(("idx", idx))
    _same_cuda_device([("q", q), ("k", k), ("v", v)] + extra)
    desc = decode_desc(q, k, group_map, scale, pooled)
    out = torch.empty_like(q) if out is None else out
    idx = torch.empty(B, H, topk, dtype=torch.int32, device=q.device) if idx is None else idx
    scores = torch.empty(B, H, N, dtype=torch.float32, device=q.device) if return_scores else None
    ws, buf = _ws(ws, q.device, workspace_size(desc, topk, DECODE), stream)
    fn, name = ((_lib.kascade_anchor_decode_fused, "kascade_anchor_decode_fused") if fused
                else (_lib.kascade_anchor_decode, "kascade_anchor_decode"))
    _check(fn(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), int(topk), _ptr(out), _ptr(idx),
              _ptr(scores), _ptr(buf), buf.numel(), _stream(stream)), name)
    return (out, idx, scores) if return_scores else (out, idx)


def reuse_decode(q, k, v, idx, group_map=None, scale=None, out=None, ws=None, stream=None,
                 pooled=False):
    """Reuse layer over saved sets idx [B,Hq,topk] (pooled: [B,Hkv,topk]; int32, ascending)."""
    B, Hq, Hkv, _, _ = _attn_inputs(q, k, v, prefill=False)
    if not isinstance(idx, torch.Tensor) or idx.dim() != 3:
        raise ValueError("idx: expected an int32 tensor [B,H,topk]")
    topk = idx.shape[-1]
    _expect(idx, "idx", (B, Hkv if pooled else Hq, topk), torch.int32)
    extra = [("idx", idx)]
    if out is not None:
        _expect(out, "out", q.shape, q.dtype)
        extra.append(("out", out))
    _same_cuda_device([("q", q), ("k", k), ("v", v)] + extra)
    desc = decode_desc(q, k, group_map, scale, pooled)
    out = torch.empty_like(q) if out is None else out
    ws, buf = _ws(ws, q.device, workspace_size(desc, topk, DECODE), stream)
    _check(_lib.kascade_reuse_decode(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), int(topk),
                                     _ptr(idx), _ptr(out), _ptr(buf), buf.numel(), _stream(stream)),
           "kascade_reuse_decode")
    return out


def anchor_decode_shard(q, k, v, key_offset, topk, group_map=None, scale=None, ws=None,
                        stream=None):
    """One shard of a KV cache split along the key axis: k/v [B,Hkv,N_s,d] hold
    global positions key_offset .. key_offset + N_s - 1. Returns the shard's
    partials (out [B,Hq,d], lse [B,Hq] fp32, cand_idx [B,Hq,topk] int32 global
    positions ascending, cand_scores [B,Hq,topk] fp32 logits)."""
    B, Hq, _, N, _ = _attn_inputs(q, k, v, prefill=False)
    _same_cuda_device([("q", q), ("k", k), ("v", v)])
    if not (1 <= int(topk) <= N) or int(key_offset) < 0:
        raise ValueError("topk must lie in [1, N_s] and key_offset must be >= 0")
    desc = decode_desc(q, k, group_map, scale)
    out = torch.empty_like(q)
    lse = torch.empty(B, Hq, dtype=torch.float32, device=q.device)
    cand_idx = torch.empty(B, Hq, topk, dtype=torch.int32, device=q.device)
    cand_scores = torch.empty(B, Hq, topk, dtype=torch.float32, device=q.device)
    ws, buf = _ws(ws, q.device, workspace_size(desc, topk, DECODE), stream)
    _check(_lib.kascade_anchor_decode_shard(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v),
                                            int(key_offset), int(topk), _ptr(out), _ptr(lse),
                                            _ptr(cand_idx), _ptr(cand_scores), _ptr(buf),
                                            buf.numel(), _stream(stream)),
           "kascade_anchor_decode_shard")
    return out, lse, cand_idx, cand_scores


def merge_decode_shards(outs, lses, cand_idx, cand_scores, n_kv_heads=None, kv_len=None,
                        ws=None, stream=None):
    """Merge S shards' partials stacked in key order: outs [S,B,Hq,d], lses
    [S,B,Hq] fp32, cand_idx [S,B,Hq,topk] int32, cand_scores [S,B,Hq,topk]
    fp32. Returns (out [B,Hq,d], idx [B,Hq,topk] ascending global positions).
    kv_len (the total keys, for the range check of the candidates) defaults
    to the largest candidate position + 1; n_kv_heads to Hq (the merge does
    not read K or V)."""
    if not isinstance(outs, torch.Tensor) or outs.dim() != 4:
        raise ValueError("outs: expected a tensor [S,B,Hq,d]")
    S, B, Hq, d = outs.shape
    if not isinstance(cand_idx, torch.Tensor) or cand_idx.dim() != 4:
        raise ValueError("cand_idx: expected an int32 tensor [S,B,Hq,topk]")
    topk = cand_idx.shape[-1]
    _expect(lses, "lses", (S, B, Hq), torch.float32)
    _expect(cand_idx, "cand_idx", (S, B, Hq, topk), torch.int32)
    _expect(cand_scores, "cand_scores", (S, B, Hq, topk), torch.float32)
    _expect(outs, "outs", (S, B, Hq, d), outs.dtype)
    _same_cuda_device([("outs", outs), ("lses", lses), ("cand_idx", cand_idx),
                       ("cand_scores", cand_scores)])
    if kv_len is None:
        kv_len = int(cand_idx.max().item()) + 1
    hkv = Hq if n_kv_heads is None else int(n_kv_heads)
    desc = make_desc(B, Hq, hkv, d, int(kv_len), _dtype_code(outs))
    out = torch.empty(B, Hq, d, dtype=outs.dtype, device=outs.device)
    idx = torch.empty(B, Hq, topk, dtype=torch.int32, device=outs.device)
    n = _lib.kascade_merge_workspace_size(ctypes.byref(desc), int(S), int(topk))
    if n == 0:
        raise KascadeError(INVALID_ARG, "kascade_merge_workspace_size")
    ws, buf = _ws(ws, outs.device, n, stream)
    _check(_lib.kascade_merge_decode_shards(ctypes.byref(desc), int(S), _ptr(outs), _ptr(lses),
                                            _ptr(cand_idx), _ptr(cand_scores), int(topk),
                                            _ptr(out), _ptr(idx), _ptr(buf), buf.numel(),
                                            _stream(stream)), "kascade_merge_decode_shards")
    return out, idx


def topk(scores, k, out=None, ws=None, stream=None):
    """Exact Top-k of fp32 rows [rows, n] -> int32 [rows, k] ascending."""
    if not isinstance(scores, torch.Tensor) or scores.dim() != 2:
        raise ValueError("scores: expected an fp32 tensor [rows, n]")
    rows, n = scores.shape
    _expect(scores, "scores", (rows, n), torch.float32)
    named = [("scores", scores)]
    if out is not None:
        _expect(out, "out", (rows, int(k)), torch.int32)
        named.append(("out", out))
    _same_cuda_device(named)
    out = torch.empty(rows, k, dtype=torch.int32, device=scores.device) if out is None else out
    ws, buf = _ws(ws, scores.device, 256, stream)
    _check(_lib.kascade_topk(_ptr(scores), rows, n, int(k), _ptr(out), _ptr(buf), buf.numel(),
                             _stream(stream)), "kascade_topk")
    return out


# ----------------------------------------------------------------- prefill --

def n_tiles(n: int) -> int:
    return (n + TILE - 1) // TILE


def dense_prefill(q, k, v, group_map=None, scale=None, out=None, ws=None, stream=None):
    """Causal exact attention: q [B,Hq,N,d], k/v [B,Hkv,N,d] (bf16)."""
    _attn_inputs(q, k, v, prefill=True)
    if out is not None:
        _expect(out, "out", q.shape, q.dtype)
    _same_cuda_device([("q", q), ("k", k), ("v", v)] + ([("out", out)] if out is not None else []))
    desc = prefill_desc(q, k, group_map, scale)
    out = torch.empty_like(q) if out is None else out
    ws, buf = _ws(ws, q.device, workspace_size(desc, 1, PREFILL), stream)
    _check(_lib.kascade_dense_prefill(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(out),
                                      _ptr(buf), buf.numel(), _stream(stream)), "kascade_dense_prefill")
    return out


def packed_tile_len(n: int) -> int:
    """Length of one (sequence, head) row of packed tile weights: sum_t L_t."""
    nt = n_tiles(n)
    return 64 * (nt - 1) * nt + n


def packed_tile_offset(t: int) -> int:
    """Offset of tile t's weights in a packed row (64 t (t + 1))."""
    return 64 * t * (t + 1)


def anchor_prefill(q, k, v, topk, group_map=None, scale=None, out=None, idx=None, ws=None,
                   stream=None, pooled=False, return_weights=False):
    """Anchor layer, prefill: (out, idx [B,H,nT,topk] int32, -1 padded), H = Hq or,
    pooled, Hkv. With return_weights, also the fp32 tile weights the selection
    ranked, packed [B,H,packed_tile_len(N)] (tile t at packed_tile_offset(t),
    L_t = min(N, 128(t+1)) entries): (out, idx, weights)."""
    B, Hq, Hkv, N, _ = _attn_inputs(q, k, v, prefill=True)
    H = Hkv if pooled else Hq
    extra = []
    if out is not None:
        _expect(out, "out", q.shape, q.dtype)
        extra.append(("out", out))
    if idx is not None:
        _expect(idx, "idx", (B, H, n_tiles(N), topk), torch.int32)
        extra.append(("idx", idx))
    _same_cuda_device([("q", q), ("k", k), ("v", v)] + extra)
    desc = prefill_desc(q, k, group_map, scale, pooled)
    out = torch.empty_like(q) if out is None else out
    if idx is None:
        idx = torch.empty(B, H, n_tiles(N), topk, dtype=torch.int32, device=q.device)
    wts = (torch.empty(B, H, packed_tile_len(N), dtype=torch.float32, device=q.device)
           if return_weights else None)
    ws, buf = _ws(ws, q.device, workspace_size(desc, topk, PREFILL), stream)
    _check(_lib.kascade_anchor_prefill(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), int(topk),
                                       _ptr(out), _ptr(idx), _ptr(wts), _ptr(buf), buf.numel(),
                                       _stream(stream)), "kascade_anchor_prefill")
    return (out, idx, wts) if return_weights else (out, idx)


def reuse_prefill(q, k, v, idx, group_map=None, scale=None, out=None, ws=None, stream=None,
                  pooled=False):
    """Reuse layer, prefill, over saved tile sets idx [B,Hq,nT,topk] (pooled: [B,Hkv,nT,topk])."""
    B, Hq, Hkv, N, _ = _attn_inputs(q, k, v, prefill=True)
    if not isinstance(idx, torch.Tensor) or idx.dim() != 4:
        raise ValueError("idx: expected an int32 tensor [B,H,nT,topk]")
    topk = idx.shape[-1]
    _expect(idx, "idx", (B, Hkv if pooled else Hq, n_tiles(N), topk), torch.int32)
    extra = [("idx", idx)]
    if out is not None:
        _expect(out, "out", q.shape, q.dtype)
        extra.append(("out", out))
    _same_cuda_device([("q", q), ("k", k), ("v", v)] + extra)
    desc = prefill_desc(q, k, group_map, scale, pooled)
    out = torch.empty_like(q) if out is None else out
    ws, buf = _ws(ws, q.device, workspace_size(desc, topk, PREFILL), stream)
    _check(_lib.kascade_reuse_prefill(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), int(topk),
                                      _ptr(idx), _ptr(out), _ptr(buf), buf.numel(),
                                      _stream(stream)), "kascade_reuse_prefill")
    return out


# ------------------------------------------------------------------- stack --

def run_stack(mode, qs, ks, vs, topk, anchors, group_map=None, scale=None, outs=None,
              idx_buf=None, ws=None, stream=None, layer_events=None, pooled=False):
    """Run a layer stack; returns (outs, idx_buf). mode: DECODE or PREFILL.

    layer_events: optional list of torch.cuda.Event (timing enabled), one per
    layer, recorded on the stream after that layer's launches. pooled: one
    index set per KV head."""
    if mode not in (DECODE, PREFILL):
        raise ValueError("mode must be DECODE or PREFILL")
    L = len(qs)
    (B, Hq, Hkv, N, _), dev = _layers(qs, ks, vs, prefill=(mode == PREFILL))
    H = Hkv if pooled else Hq
    if mode == DECODE:
        desc = decode_desc(qs[0], ks[0], group_map, scale, pooled)
        shape = (B, H, topk)
    else:
        desc = prefill_desc(qs[0], ks[0], group_map, scale, pooled)
        shape = (B, H, n_tiles(N), topk)
    if outs is not None:
        if len(outs) != L:
            raise ValueError("outs: one tensor per layer (got %d for %d layers)" % (len(outs), L))
        _all_like(outs, "outs", qs[0].shape, qs[0].dtype, dev)
    if idx_buf is not None:
        _expect(idx_buf, "idx_buf", shape, torch.int32)
        _same_cuda_device([("qs[0]", qs[0]), ("idx_buf", idx_buf)])
    if layer_events is not None and len(layer_events) != L:
        raise ValueError("layer_events: one event per layer")
    outs = [torch.empty_like(q) for q in qs] if outs is None else outs
    if idx_buf is None:
        idx_buf = torch.empty(shape, dtype=torch.int32, device=dev)
    ws, buf = _ws(ws, dev, workspace_size(desc, topk, mode), stream)
    arr = lambda ts: (ctypes.c_void_p * L)(*[t.data_ptr() for t in ts])
    an = (ctypes.c_int32 * max(1, len(anchors)))(*[int(a) for a in anchors])
    if layer_events is None:
        _check(_lib.kascade_run_stack(ctypes.byref(desc), int(mode), L, arr(qs), arr(ks), arr(vs),
                                      int(topk), an, len(anchors), arr(outs), _ptr(idx_buf),
                                      _ptr(buf), buf.numel(), _stream(stream)), "kascade_run_stack")
    else:
        ev = (ctypes.c_void_p * L)(*[e.cuda_event for e in layer_events])
        _check(_lib.kascade_run_stack_profiled(ctypes.byref(desc), int(mode), L, arr(qs), arr(ks),
                                               arr(vs), int(topk), an, len(anchors), arr(outs),
                                               _ptr(idx_buf), _ptr(buf), buf.numel(),
                                               _stream(stream), ev), "kascade_run_stack_profiled")
    return outs, idx_buf


def kascade_attention(qs, ks, vs, topk, anchors, group_map=None, scale=None, pooled=False,
                      ws=None, stream=None):
    """One call over a layer stack, in the form the Kascade pages describe
    (euno.news summary, Practical Implications): per-layer lists qs, ks, vs,
    the Top-k size and the anchor layers. 3-D queries [B,Hq,d] are decode,
    4-D [B,Hq,N,d] causal prefill. Anchor layers compute exact attention and
    refresh the index sets, the layers after them reuse those sets, and
    layers before the first anchor run dense. Returns the per-layer outputs."""
    if len(qs) == 0:
        raise ValueError("qs: at least one layer")
    mode = DECODE if qs[0].dim() == 3 else PREFILL
    outs, _ = run_stack(mode, qs, ks, vs, topk, list(anchors), group_map=group_map, scale=scale,
                        ws=ws, stream=stream, pooled=pooled)
    return outs


# ------------------------------------------------- paged 4-bit key/value cache --
# The pages (one uint8 tensor per layer, qcache_alloc) hold num_blocks blocks of
# block_size tokens, [num_blocks, Hkv, block_size/16, 18*d]; a block table
# [B, max_blocks] lists each sequence's blocks and kv_lens [B] its cached
# tokens. Number format, layout and error behaviour: include/kascade.h. stream=:
# the torch.cuda.Stream to work on instead of the current one; its inputs have
# to be ready on it, and its outputs belong to it.

def qcache_alloc(num_blocks, n_kv_heads, head_dim, block_size=64, device="cuda"):
    """Zeroed pages of one layer: uint8 [num_blocks, Hkv, block_size/16, 18*d]."""
    geo = QCache(int(block_size), int(num_blocks), 1, 0.0, 0.0)
    n = _lib.kascade_qcache_bytes(ctypes.byref(geo), int(n_kv_heads), int(head_dim))
    if n == 0:
        raise KascadeError(INVALID_ARG, "kascade_qcache_bytes")
    return torch.zeros(int(num_blocks), int(n_kv_heads), int(block_size) // 16, 18 * int(head_dim),
                       dtype=torch.uint8, device=device)


# A decode step's calls take a few microseconds on the GPU, so the host side is
# kept short: each tensor passes one combined test and gets the detailed one
# only when that fails, and the structures that depend on sizes alone are built
# once per geometry.

def _fits(t, name, shape, dtype, dev):
    """One tensor's type, shape, dtype, device and contiguity."""
    if not (isinstance(t, torch.Tensor) and t.shape == shape and t.dtype is dtype
            and t.device == dev and t.is_contiguous()):
        _expect(t, name, shape, dtype)
        raise ValueError("%s: on %s, expected %s" % (name, t.device, dev))


def _cuda(t, name):
    """The CUDA device of a call's first tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s: expected a torch.Tensor" % name)
    dev = t.device
    if dev.type != _DEVICE_TYPE:
        raise ValueError("%s: on %s; the library takes CUDA device tensors" % (name, dev))
    return dev


# torch.cuda.current_device, current_stream and is_current_stream_capturing
# without their wrapper objects (each costs a microsecond or two); these
# themselves where torch does not have the functions behind them
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                              lambda index: torch.cuda.current_stream(index).cuda_stream)
_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing",
                     torch.cuda.is_current_stream_capturing)


def _elsewhere(index, stream):
    """Whether a call whose tensors are on CUDA device `index` (-1: not on one)
    has to switch to another device or stream first (_on)."""
    return stream is not None or (index >= 0 and index != _current_device())


def _on(dev, stream, *tensors):
    """Context in which the tensors' device and the call's stream are current,
    so that what the call allocates belongs to that stream; inside it the call
    is made again without a stream. The stream is noted on the call's tensors
    (None among them: not given), so that the memory of one that the caller drops
    is not given out again while the stream still reads or writes it."""
    if dev.type != "cuda":      # only reachable with a stand-in library
        return contextlib.nullcontext()
    if stream is None:
        return torch.cuda.device(dev)
    if stream.device != dev:
        raise ValueError("stream: on %s, expected %s" % (stream.device, dev))
    for t in tensors:
        if t is not None:
            t.record_stream(stream)
    return torch.cuda.stream(stream)


def _raw_stream(index):
    return _current_raw_stream(index) if index >= 0 else None


def _qws(ws, dev, index, nbytes):
    """The workspace buffer of a cache call (by default the current stream's
    own, default_workspace). A captured call needs a workspace
    of its own, large enough already: a graph keeps its address, so the
    shared default one (which grows) or one grown inside the capture would be
    gone when the graph is replayed."""
    if index >= 0 and _capturing():
        if ws is None or ws.buf is None or ws.buf.numel() < nbytes:
            raise ValueError("a captured call needs ws=Workspace(device), sized before the capture "
                             "(run the call once with it)")
        ws.captured = True
    if ws is None:
        raw = _current_raw_stream(index)
        ws = _default_ws.get((index, raw) if raw else index) or _workspace_of(index, raw)
    buf = ws.buf
    if buf is None or buf.numel() < nbytes:
        buf = ws.get(nbytes)
    if buf.get_device() != index:
        raise ValueError("ws: on %s, expected %s" % (buf.device, dev))
    return buf


def _pages(pages, name="pages"):
    """Validated (num_blocks, Hkv, block_size, d) of one layer's pages."""
    if not isinstance(pages, torch.Tensor) or pages.dim() != 4:
        raise ValueError("%s: expected a uint8 tensor [num_blocks, Hkv, block_size/16, 18*d]" % name)
    nb, hkv, groups, size = pages.shape
    if size != 2304 and size != 1152:
        raise ValueError("%s: last axis %d, expected 18*d with d 64 or 128" % (name, size))
    if pages.dtype is not torch.uint8 or not pages.is_contiguous():
        _expect(pages, name, pages.shape, torch.uint8)
    return nb, hkv, groups * 16, size // 18


@functools.lru_cache(maxsize=256)
def _qgeo(block_size, num_blocks, max_blocks, k_scale, v_scale):
    """A kascade_qcache structure by value (read only), as a ctypes reference."""
    return ctypes.byref(QCache(block_size, num_blocks, max_blocks, k_scale, v_scale))


@functools.lru_cache(maxsize=256)
def _qdesc(B, Hq, Hkv, d, N, code, scale, group_map, pooled, bs, nb, width, k_scale, v_scale, topk,
           reuse):
    """Descriptor, geometry (ctypes references, read only) and workspace bytes of
    an attention call of these sizes."""
    desc = make_desc(B, Hq, Hkv, d, N, code, scale, group_map, pooled)
    geo = QCache(bs, nb, width, k_scale, v_scale)
    return ctypes.byref(desc), ctypes.byref(geo), qcache_workspace_size(desc, geo, topk, reuse)


def qcache_workspace_size(desc, geo, topk: int, reuse: bool = False) -> int:
    """Workspace bytes of a cache attention call (topk 0: dense decode); reuse: of a
    reuse layer alone, which keeps no logits."""
    name = "kascade_qcache_reuse_workspace_size" if reuse else "kascade_qcache_workspace_size"
    n = getattr(_lib, name)(ctypes.byref(desc), ctypes.byref(geo), int(topk))
    if n == 0:
        raise KascadeError(INVALID_ARG, name)
    return n


def qcache_plan(kv_lens, new_lens, block_table, free_blocks, free_count, block_size, max_new,
                kv_lens_out=None, free_count_out=None, ws=None, stream=None):
    """Block tables and slots of one step, on the device: sequence b goes from
    kv_lens[b] to max(0, kv_lens[b] + new_lens[b]) tokens, takes blocks from the
    top of the stack free_blocks [num_blocks] (free_count [1] of them valid)
    and gives back those it no longer needs. block_table [B, max_blocks] and
    free_blocks are updated in place. Returns (slot_map [max_new], cu_new
    [B+1], kv_lens_out [B], free_count_out [1]), all int32; the last two may
    be given (kv_lens and free_count themselves included)."""
    i32 = torch.int32
    if not (isinstance(block_table, torch.Tensor) and isinstance(kv_lens, torch.Tensor)
            and isinstance(new_lens, torch.Tensor) and isinstance(free_blocks, torch.Tensor)
            and isinstance(free_count, torch.Tensor) and block_table.dim() == 2
            and free_blocks.dim() == 1 and block_table.dtype is i32 and kv_lens.dtype is i32
            and new_lens.dtype is i32 and free_blocks.dtype is i32 and free_count.dtype is i32
            and kv_lens.shape == block_table.shape[:1] and new_lens.shape == kv_lens.shape
            and free_count.shape == (1,) and block_table.is_contiguous()
            and kv_lens.is_contiguous() and new_lens.is_contiguous()
            and free_blocks.is_contiguous() and block_table.device.type == _DEVICE_TYPE
            and kv_lens.device == block_table.device and new_lens.device == block_table.device
            and free_blocks.device == block_table.device
            and free_count.device == block_table.device):
        dev = _cuda(block_table, "block_table")      # what is wrong, in words
        if block_table.dim() != 2:
            raise ValueError("block_table: expected an int32 tensor [B, max_blocks]")
        if not isinstance(free_blocks, torch.Tensor) or free_blocks.dim() != 1:
            raise ValueError("free_blocks: expected an int32 tensor [num_blocks]")
        _fits(block_table, "block_table", block_table.shape, i32, dev)
        _fits(kv_lens, "kv_lens", block_table.shape[:1], i32, dev)
        _fits(new_lens, "new_lens", block_table.shape[:1], i32, dev)
        _fits(free_blocks, "free_blocks", free_blocks.shape, i32, dev)
        _fits(free_count, "free_count", (1,), i32, dev)
    dev = block_table.device
    B, width = block_table.shape
    if kv_lens_out is not None:
        _fits(kv_lens_out, "kv_lens_out", (B,), i32, dev)
    if free_count_out is not None:
        _fits(free_count_out, "free_count_out", (1,), i32, dev)
    max_new = int(max_new)
    geo = _qgeo(int(block_size), free_blocks.shape[0], width, 0.0, 0.0)
    index = block_table.get_device()
    if _elsewhere(index, stream):
        with _on(dev, stream, kv_lens, new_lens, block_table, free_blocks, free_count,
                 kv_lens_out, free_count_out):
            return qcache_plan(kv_lens, new_lens, block_table, free_blocks, free_count, block_size,
                               max_new, kv_lens_out, free_count_out, ws)
    # one by one: an allocation and three views of it take 2 us longer
    slots = torch.empty(max(max_new, 0), dtype=i32, device=dev)
    cu = torch.empty(B + 1, dtype=i32, device=dev)
    lens = torch.empty(B, dtype=i32, device=dev) if kv_lens_out is None else kv_lens_out
    count = torch.empty(1, dtype=i32, device=dev) if free_count_out is None else free_count_out
    buf = _qws(ws, dev, index, 256)
    _check(_lib.kascade_qcache_plan(geo, B, kv_lens.data_ptr(), new_lens.data_ptr(),
                                    block_table.data_ptr(), free_blocks.data_ptr(),
                                    free_count.data_ptr(), lens.data_ptr(), count.data_ptr(),
                                    cu.data_ptr(), slots.data_ptr(), max_new, buf.data_ptr(),
                                    buf.numel(), _raw_stream(index)), "kascade_qcache_plan")
    return slots, cu, lens, count


_I64x4 = ctypes.c_int64 * 4
_ROW_CODES = {torch.bfloat16: (BF16, 8), torch.float32: (F32, 4)}   # code, elements per 16 bytes


def _row_strides(t, name, shape, dtype, dev, unit):
    """Token and head strides of rows t [T, Hkv, d], which must be contiguous and
    start on 16-byte boundaries (strides of axes of length 1 do not matter)."""
    if not (isinstance(t, torch.Tensor) and t.shape == shape and t.dtype is dtype
            and t.device == dev):
        if not isinstance(t, torch.Tensor):
            raise TypeError("%s: expected a torch.Tensor" % name)
        if t.shape != shape:
            raise ValueError("%s: shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
        if t.dtype is not dtype:
            raise TypeError("%s: dtype %s, expected %s" % (name, t.dtype, dtype))
        raise ValueError("%s: on %s, expected %s" % (name, t.device, dev))
    tok, head, one = t.stride()
    if shape[0] <= 1 or shape[1] <= 1:
        tok, head = tok if shape[0] > 1 else 0, head if shape[1] > 1 else 0
    if shape[0] and (one != 1 or tok % unit or head % unit or t.data_ptr() % 16):
        raise ValueError("%s: rows must be contiguous and start on 16-byte boundaries" % name)
    return tok, head


def _slots(slot_map, dev):
    if not isinstance(slot_map, torch.Tensor) or slot_map.dim() != 1:
        raise ValueError("slot_map: expected an int32 tensor [T]")
    _fits(slot_map, "slot_map", slot_map.shape, torch.int32, dev)
    return slot_map.shape[0]


def qcache_append(k, v, slot_map, pages, k_scale=1.0, v_scale=1.0, ws=None, stream=None):
    """Quantise rows k, v [T, Hkv, d] (bf16 or fp32; any token and head strides,
    so a prefill layer's k[b].transpose(0, 1) is taken as it is) into the slots
    slot_map [T] int32 (distinct; negative: skipped) of pages, in place."""
    nb, hkv, bs, d = _pages(pages)
    dev = _cuda(pages, "pages")
    T = _slots(slot_map, dev)
    if not isinstance(k, torch.Tensor) or k.dtype not in _ROW_CODES:
        raise TypeError("k: expected a bfloat16 or float32 tensor")
    code, unit = _ROW_CODES[k.dtype]
    kt, kh = _row_strides(k, "k", (T, hkv, d), k.dtype, dev, unit)
    vt, vh = _row_strides(v, "v", (T, hkv, d), k.dtype, dev, unit)
    geo = _qgeo(bs, nb, 1, float(k_scale), float(v_scale))
    index = pages.get_device()
    if _elsewhere(index, stream):
        with _on(dev, stream, k, v, slot_map, pages):
            return qcache_append(k, v, slot_map, pages, k_scale, v_scale, ws)
    buf = _qws(ws, dev, index, 256)
    _check(_lib.kascade_qcache_append(geo, hkv, d, code, k.data_ptr(), v.data_ptr(),
                                      _I64x4(kt, kh, vt, vh),
                                      slot_map.data_ptr(), T, pages.data_ptr(),
                                      buf.data_ptr(), buf.numel(), _raw_stream(index)),
           "kascade_qcache_append")
    return pages


def qcache_read(pages, slot_map, dtype=torch.bfloat16, k_scale=1.0, v_scale=1.0, k=None, v=None,
                ws=None, stream=None):
    """The stored values of slots slot_map [T] int32 as (k, v) [T, Hkv, d] (bf16
    or fp32; zeros for a negative slot). k, v: outputs to fill instead, of any
    token and head strides whose rows do not overlap."""
    nb, hkv, bs, d = _pages(pages)
    dev = _cuda(pages, "pages")
    T = _slots(slot_map, dev)
    if (k is None) != (v is None):
        raise ValueError("k, v: give both outputs or neither")
    if k is not None:
        if not isinstance(k, torch.Tensor):
            raise TypeError("k: expected a torch.Tensor")
        dtype = k.dtype
    if dtype not in _ROW_CODES:
        raise TypeError("rows are read as bfloat16 or float32")
    code, unit = _ROW_CODES[dtype]
    shape = (T, hkv, d)
    if k is None:
        strides = (hkv * d, d, hkv * d, d)
    else:
        strides = (_row_strides(k, "k", shape, dtype, dev, unit) +
                   _row_strides(v, "v", shape, dtype, dev, unit))
        if T and any(n > 1 and st == 0 for st, n in zip(strides, (T, hkv, T, hkv))):
            raise ValueError("k, v: output rows must not overlap")
    geo = _qgeo(bs, nb, 1, float(k_scale), float(v_scale))
    index = pages.get_device()
    if _elsewhere(index, stream):
        with _on(dev, stream, pages, slot_map, k, v):
            return qcache_read(pages, slot_map, dtype, k_scale, v_scale, k, v, ws)
    ok = torch.empty(shape, dtype=dtype, device=dev) if k is None else k
    ov = torch.empty(shape, dtype=dtype, device=dev) if v is None else v
    buf = _qws(ws, dev, index, 256)
    _check(_lib.kascade_qcache_read(geo, hkv, d, code, pages.data_ptr(), slot_map.data_ptr(),
                                    T, ok.data_ptr(), ov.data_ptr(),
                                    _I64x4(*strides), buf.data_ptr(),
                                    buf.numel(), _raw_stream(index)), "kascade_qcache_read")
    return ok, ov


def _qattn(q, pages, block_table, kv_lens, kv_len, group_map, scale, k_scale, v_scale, pooled, topk,
           out, reuse=False):
    """Checks one attention call's common tensors; returns (descriptor and
    geometry references, workspace bytes, (B, Hq, Hkv, N), device)."""
    nb, hkv, bs, d = _pages(pages)
    dev = pages.device
    if not (dev.type == _DEVICE_TYPE and isinstance(q, torch.Tensor)
            and isinstance(block_table, torch.Tensor) and isinstance(kv_lens, torch.Tensor)
            and q.dim() == 3 and block_table.dim() == 2 and q.dtype in _ROW_CODES
            and q.shape[2] == d and q.device == dev and q.is_contiguous()
            and block_table.shape[0] == q.shape[0] and block_table.dtype is torch.int32
            and block_table.device == dev and block_table.is_contiguous()
            and kv_lens.shape == q.shape[:1] and kv_lens.dtype is torch.int32
            and kv_lens.device == dev and kv_lens.is_contiguous()):
        _cuda(pages, "pages")        # what is wrong, in words
        if not isinstance(q, torch.Tensor) or q.dim() != 3:
            raise ValueError("q: expected a tensor [B,Hq,d]")
        _dtype_code(q)
        if q.shape[2] != d:
            raise ValueError("q: head_dim %d, the pages hold %d" % (q.shape[2], d))
        _fits(q, "q", q.shape, q.dtype, dev)
        if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
            raise ValueError("block_table: expected an int32 tensor [B, max_blocks]")
        _fits(block_table, "block_table", (q.shape[0], block_table.shape[1]), torch.int32, dev)
        _fits(kv_lens, "kv_lens", (q.shape[0],), torch.int32, dev)
    B, Hq, _ = q.shape
    width = block_table.shape[1]
    if out is not None:
        _fits(out, "out", q.shape, q.dtype, dev)
    N = width * bs if kv_len is None else int(kv_len)
    desc, geo, nbytes = _qdesc(B, Hq, hkv, d, N, _ROW_CODES[q.dtype][0],
                               0.0 if scale is None else float(scale),
                               None if group_map is None else tuple(int(x) for x in group_map),
                               bool(pooled), bs, nb, width, float(k_scale), float(v_scale), topk,
                               reuse)
    return desc, geo, nbytes, (B, Hq, hkv, N), dev


def qcache_dense_decode(q, pages, block_table, kv_lens, kv_len=None, group_map=None, scale=None,
                        k_scale=1.0, v_scale=1.0, return_scores=False, out=None, ws=None,
                        stream=None):
    """Exact decode attention q [B,Hq,d] over the cached tokens of each sequence
    -> out [B,Hq,d], or (out, scores [B,Hq,kv_len] fp32 logits, -inf behind
    the last token). kv_len: the longest length any kv_lens[b] may have
    (default: what the block table can hold). The workspace and the limits of a
    call go by kv_len, not by the lengths themselves: give it where the table is
    wide."""
    desc, geo, nbytes, (B, Hq, _, N), dev = _qattn(q, pages, block_table, kv_lens, kv_len,
                                                   group_map, scale, k_scale, v_scale, False, 0,
                                                   out)
    index = pages.get_device()
    if _elsewhere(index, stream):
        with _on(dev, stream, q, pages, block_table, kv_lens, out):
            return qcache_dense_decode(q, pages, block_table, kv_lens, kv_len, group_map, scale,
                                       k_scale, v_scale, return_scores, out, ws)
    o = torch.empty_like(q) if out is None else out
    scores = (torch.empty(B, Hq, N, dtype=torch.float32, device=dev) if return_scores
              else None)
    buf = _qws(ws, dev, index, nbytes)
    _check(_lib.kascade_qcache_dense_decode(desc, geo, q.data_ptr(), pages.data_ptr(),
                                            block_table.data_ptr(), kv_lens.data_ptr(),
                                            o.data_ptr(),
                                            scores.data_ptr() if return_scores else None,
                                            buf.data_ptr(), buf.numel(), _raw_stream(index)),
           "kascade_qcache_dense_decode")
    return (o, scores) if return_scores else o


def qcache_anchor_decode(q, pages, block_table, kv_lens, topk, kv_len=None, group_map=None,
                         scale=None, k_scale=1.0, v_scale=1.0, return_scores=False, out=None,
                         idx=None, ws=None, stream=None, pooled=False):
    """Anchor layer over the cache: (out [B,Hq,d], idx [B,H,topk] int32[, scores
    [B,H,kv_len] fp32]), as anchor_decode; rows of a sequence with fewer than
    topk tokens end in -1 entries."""
    topk = int(topk)
    desc, geo, nbytes, (B, Hq, hkv, N), dev = _qattn(q, pages, block_table, kv_lens, kv_len,
                                                     group_map, scale, k_scale, v_scale, pooled,
                                                     max(topk, 1), out)
    H = hkv if pooled else Hq
    if idx is not None:
        _fits(idx, "idx", (B, H, topk), torch.int32, dev)
    index = pages.get_device()
    if _elsewhere(index, stream):
        with _on(dev, stream, q, pages, block_table, kv_lens, out, idx):
            return qcache_anchor_decode(q, pages, block_table, kv_lens, topk, kv_len, group_map, scale,
                                        k_scale, v_scale, return_scores, out, idx, ws,
                                        pooled=pooled)
    o = torch.empty_like(q) if out is None else out
    ix = torch.empty(B, H, topk, dtype=torch.int32, device=dev) if idx is None else idx
    scores = torch.empty(B, H, N, dtype=torch.float32, device=dev) if return_scores else None
    buf = _qws(ws, dev, index, nbytes)
    _check(_lib.kascade_qcache_anchor_decode(desc, geo, q.data_ptr(), pages.data_ptr(),
                                             block_table.data_ptr(), kv_lens.data_ptr(), topk,
                                             o.data_ptr(), ix.data_ptr(),
                                             scores.data_ptr() if return_scores else None,
                                             buf.data_ptr(), buf.numel(), _raw_stream(index)),
           "kascade_qcache_anchor_decode")
    return (o, ix, scores) if return_scores else (o, ix)


def qcache_reuse_decode(q, pages, block_table, kv_lens, idx, kv_len=None, group_map=None,
                        scale=None, k_scale=1.0, v_scale=1.0, out=None, ws=None, stream=None,
                        pooled=False):
    """Reuse layer over the cache and saved sets idx [B,Hq,topk] (pooled:
    [B,Hkv,topk]; int32, ascending, -1 behind the last entry)."""
    if not isinstance(idx, torch.Tensor) or idx.dim() != 3:
        raise ValueError("idx: expected an int32 tensor [B,H,topk]")
    topk = idx.shape[2]
    desc, geo, nbytes, (B, Hq, hkv, _), dev = _qattn(q, pages, block_table, kv_lens, kv_len,
                                                     group_map, scale, k_scale, v_scale, pooled,
                                                     max(topk, 1), out, reuse=True)
    _fits(idx, "idx", (B, hkv if pooled else Hq, topk), torch.int32, dev)
    index = pages.get_device()
    if _elsewhere(index, stream):
        with _on(dev, stream, q, pages, block_table, kv_lens, idx, out):
            return qcache_reuse_decode(q, pages, block_table, kv_lens, idx, kv_len, group_map, scale,
                                       k_scale, v_scale, out, ws, pooled=pooled)
    o = torch.empty_like(q) if out is None else out
    buf = _qws(ws, dev, index, nbytes)
    _check(_lib.kascade_qcache_reuse_decode(desc, geo, q.data_ptr(), pages.data_ptr(),
                                            block_table.data_ptr(), kv_lens.data_ptr(), topk,
                                            idx.data_ptr(), o.data_ptr(), buf.data_ptr(),
                                            buf.numel(), _raw_stream(index)),
           "kascade_qcache_reuse_decode")
    return o


def qcache_run_stack(qs, pages, block_table, kv_lens, topk, anchors, new_ks=None, new_vs=None,
                     new_lens=None, free_blocks=None, free_count=None, slot_map=None, cu_new=None,
                     kv_len=None, group_map=None, scale=None, k_scale=1.0, v_scale=1.0, outs=None,
                     idx_buf=None, ws=None, stream=None, pooled=False):
    """One decode step over a layer stack on paged 4-bit caches: per-layer lists
    qs [B,Hq,d] and pages, and optionally the step's new rows new_ks, new_vs
    [T,Hkv,d]. With new_lens [B] (and free_blocks, free_count) the step first
    plans its blocks and slots, updating block_table, kv_lens, free_blocks and
    free_count in place; without, new rows go to slot_map [T] and kv_lens
    counts them already. Then every layer appends its rows and runs as anchor,
    reuse or (before the first anchor) dense layer. Returns (outs, idx_buf)."""
    L = len(qs)
    if L < 1 or len(pages) != L:
        raise ValueError("qs, pages: one tensor per layer each (got %d, %d)" % (L, len(pages)))
    if (new_ks is None) != (new_vs is None):
        raise ValueError("new_ks, new_vs: give both or neither")
    if new_ks is not None and (len(new_ks) != L or len(new_vs) != L):
        raise ValueError("new_ks, new_vs: one tensor per layer")
    if (new_lens is None) != (free_blocks is None) or (new_lens is None) != (free_count is None):
        raise ValueError("new_lens, free_blocks, free_count: give all or none")
    if new_lens is None and new_ks is not None and slot_map is None:
        raise ValueError("new rows need new_lens (a plan) or slot_map")
    topk = int(topk)
    desc, geo, nbytes, (B, Hq, hkv, N), dev = _qattn(
        qs[0], pages[0], block_table, kv_lens, kv_len, group_map, scale, k_scale, v_scale, pooled,
        max(topk, 1) if len(anchors) else 0, None)
    _all_like(qs, "qs", qs[0].shape, qs[0].dtype, dev)
    _all_like(pages, "pages", pages[0].shape, torch.uint8, dev)
    T = 0
    if new_ks is not None:
        if not isinstance(new_ks[0], torch.Tensor) or new_ks[0].dim() != 3:
            raise ValueError("new_ks[0]: expected a tensor [T,Hkv,d]")
        T = new_ks[0].shape[0]
        for name, ts in (("new_ks", new_ks), ("new_vs", new_vs)):
            _all_like(ts, name, torch.Size((T, hkv, qs[0].shape[2])), qs[0].dtype, dev)
    elif slot_map is not None:
        T = slot_map.numel()
    ints = [("new_lens", new_lens, (B,)), ("slot_map", slot_map, (T,)), ("cu_new", cu_new, (B + 1,)),
            ("free_count", free_count, (1,)), ("free_blocks", free_blocks, (pages[0].shape[0],))]
    for name, t, shape in ints:
        if t is not None:
            _fits(t, name, shape, torch.int32, dev)
    H = hkv if pooled else Hq
    if outs is not None:
        if len(outs) != L:
            raise ValueError("outs: one tensor per layer (got %d for %d layers)" % (len(outs), L))
        _all_like(outs, "outs", qs[0].shape, qs[0].dtype, dev)
    if idx_buf is not None:
        _fits(idx_buf, "idx_buf", (B, H, max(topk, 1)), torch.int32, dev)
    index = qs[0].get_device()
    if _elsewhere(index, stream):
        lists = [ts for ts in (qs, pages, new_ks, new_vs, outs) if ts is not None]
        with _on(dev, stream, block_table, kv_lens, new_lens, free_blocks, free_count, slot_map,
                 cu_new, idx_buf, *(t for ts in lists for t in ts)):
            return qcache_run_stack(qs, pages, block_table, kv_lens, topk, anchors, new_ks, new_vs,
                                    new_lens, free_blocks, free_count, slot_map, cu_new, kv_len,
                                    group_map, scale, k_scale, v_scale, outs, idx_buf, ws,
                                    pooled=pooled)
    new = lambda *n: torch.empty(*n, dtype=torch.int32, device=dev)
    os_ = [torch.empty_like(q) for q in qs] if outs is None else outs
    ib = new(B, H, max(1, topk)) if idx_buf is None else idx_buf
    sm, cu = slot_map, cu_new
    if new_lens is not None:
        sm = new(T) if sm is None else sm
        cu = new(B + 1) if cu is None else cu
    addr = lambda t: None if t is None else t.data_ptr()
    step = QCacheStep(addr(block_table), addr(kv_lens), addr(new_lens), addr(free_blocks),
                      addr(free_count), addr(cu), addr(sm), T)
    buf = _qws(ws, dev, index, nbytes)
    arr = lambda ts: (ctypes.c_void_p * L)(*[t.data_ptr() for t in ts])
    an = (ctypes.c_int32 * max(1, len(anchors)))(*[int(a) for a in anchors])
    _check(_lib.kascade_qcache_run_stack(desc, geo, ctypes.byref(step), L, arr(qs),
                                         arr(new_ks) if new_ks is not None else None,
                                         arr(new_vs) if new_vs is not None else None,
                                         arr(pages), topk, an, len(anchors), arr(os_),
                                         ib.data_ptr(), buf.data_ptr(), buf.numel(),
                                         _raw_stream(index)), "kascade_qcache_run_stack")
    return os_, ib


# -------------------------------------------------------------- scheduling --

def layer_overlap(sets, n_bits, ws=None, stream=None):
    """sets: int32 [L, units, topk] on the device -> int64 counts [L, L]."""
    if not isinstance(sets, torch.Tensor) or sets.dim() != 3:
        raise ValueError("sets: expected an int32 tensor [L, units, topk]")
    L, units, k = sets.shape
    _expect(sets, "sets", (L, units, k), torch.int32)
    _same_cuda_device([("sets", sets)])
    counts = torch.empty(L, L, dtype=torch.int64, device=sets.device)
    nbytes = _lib.kascade_overlap_workspace_size(L, units, int(n_bits))
    ws, buf = _ws(ws, sets.device, nbytes, stream)
    _check(_lib.kascade_layer_overlap(_ptr(sets), L, units, k, int(n_bits), _ptr(counts),
                                      _ptr(buf), buf.numel(), _stream(stream)), "kascade_layer_overlap")
    return counts


def schedule_anchors(sim, n_anchors: int):
    """Host DP over a similarity matrix (sequence of rows); returns (anchors, objective)."""
    L = len(sim)
    flat = (ctypes.c_double * (L * L))(*[float(x) for row in sim for x in row])
    out = (ctypes.c_int32 * n_anchors)()
    obj = ctypes.c_double()
    _check(_lib.kascade_schedule_anchors(flat, L, int(n_anchors), out, ctypes.byref(obj)),
           "kascade_schedule_anchors")
    return list(out), obj.value


def calibrate(qs, ks, vs, topk, group_map=None, scale=None, ws=None, stream=None, pooled=False,
              similarity="overlap"):
    """Every layer as an anchor; returns (sim [L][L] list of lists, sets [L, B*H, topk]),
    H = Hq, or Hkv when pooled. similarity: "overlap" (Top-k set overlap) or
    "recall" (attention mass of layer l kept by layer i's set; 0 for i > l)."""
    if similarity not in ("overlap", "recall"):
        raise ValueError("similarity must be 'overlap' or 'recall'")
    recall = similarity == "recall"
    L = len(qs)
    (B, Hq, Hkv, _, _), dev = _layers(qs, ks, vs, prefill=False)
    desc = decode_desc(qs[0], ks[0], group_map, scale, pooled)
    H = Hkv if pooled else Hq
    outs = [torch.empty_like(q) for q in qs]
    sets = torch.empty(L, B * H, topk, dtype=torch.int32, device=dev)
    size_fn = (_lib.kascade_calibrate_recall_workspace_size if recall
               else _lib.kascade_calibrate_workspace_size)
    nbytes = size_fn(ctypes.byref(desc), int(topk), L)
    if nbytes == 0:
        raise KascadeError(INVALID_ARG, "calibration workspace size")
    ws, buf = _ws(ws, dev, nbytes, stream)
    arr = lambda ts: (ctypes.c_void_p * L)(*[t.data_ptr() for t in ts])
    sim = (ctypes.c_double * (L * L))()
    fn = _lib.kascade_calibrate_recall if recall else _lib.kascade_calibrate
    _check(fn(ctypes.byref(desc), L, arr(qs), arr(ks), arr(vs), int(topk), arr(outs), _ptr(sets),
              sim, _ptr(buf), buf.numel(), _stream(stream)),
           "kascade_calibrate_recall" if recall else "kascade_calibrate")
    return [[sim[i * L + j] for j in range(L)] for i in range(L)], sets
