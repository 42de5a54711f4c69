"""Thin ctypes binding of libdspark (argument marshalling only).

Every function checks shapes, dtypes, devices and contiguity of torch tensors,
allocates missing outputs and workspaces with torch, and calls the C entry
point of the same name on the current CUDA stream.  No step of the method runs
in Python.  If the library cannot be loaded the functions raise: there is no
fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math
import os
import threading
from fractions import Fraction

import torch

from . import build as _build

DSPARK_OK = 0
DSPARK_BF16 = 0
DSPARK_F32 = 1
DSPARK_F16 = 2
KV_E4M3, KV_INT8 = 0, 1
MASK_CAUSAL, MASK_FULL = 0, 1
WS_DRAFT, WS_SCHEDULE, WS_VERIFY, WS_DRAFT_RNN = 0, 1, 2, 3

FLAG_BAD_TOKEN = 1
FLAG_BAD_TEMPERATURE = 2
FLAG_BAD_VERIFY_LEN = 4
FLAG_BAD_POS_TEMP = 8
FLAG_TIMEOUT = 16
FLAG_BAD_TARGET_ROW = 32
FLAG_BAD_PAGE = 64
FLAG_BAD_LENGTH = 128
FLAG_NONFINITE = 256

EXPORTS = ("dspark_version", "dspark_last_error", "dspark_workspace_bytes", "dspark_draft_sample",
           "dspark_schedule_prefix", "dspark_schedule_policy", "dspark_verify", "dspark_read_device_flags",
           "dspark_verify_noalloc", "dspark_draft_sample_rnn", "dspark_verify_packed", "dspark_pack_target",
           "dspark_selftest_bounded_wait", "dspark_read_noalloc_flags", "dspark_selftest_philox_rate",
           "dspark_kv_append", "dspark_kv_read", "dspark_attention_workspace_bytes", "dspark_block_attention",
           "dspark_rotary_rows", "dspark_kv_append_rotary", "dspark_window_workspace_bytes", "dspark_window_attention")

_lib = None
_lock = threading.Lock()


class _CacheStruct(ctypes.Structure):
    """struct dspark_kv_cache"""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale", "flags")]
                + [(n, ctypes.c_int32) for n in ("n_pages", "n_kv_heads", "page_size", "head_dim", "format")])


class _RotaryStruct(ctypes.Structure):
    """struct dspark_rotary"""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("step", "axis")]
                + [(n, ctypes.c_int32) for n in ("n_pairs", "n_axes", "adjacent")])


class DSparkError(RuntimeError):
    def __init__(self, status, message):
        super().__init__("dspark status %d: %s" % (status, message))
        self.status = status


def library_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = True):
    """Load libdspark.so (building it first when missing or stale)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = _build.LIB
        if build_if_missing and not _build.up_to_date():
            _build.build_library()
        if not os.path.exists(path):
            raise RuntimeError("libdspark.so not built: run __graft_entry__.build()")
        L = ctypes.CDLL(path)
        vp, i32, u64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_uint64, ctypes.c_size_t
        L.dspark_version.restype = ctypes.c_int
        L.dspark_version.argtypes = []
        L.dspark_last_error.restype = ctypes.c_char_p
        L.dspark_last_error.argtypes = []
        L.dspark_workspace_bytes.restype = sz
        L.dspark_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
        L.dspark_draft_sample.restype = ctypes.c_int
        L.dspark_draft_sample.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, u64,
                                          vp, vp, vp, vp, vp, sz, vp]
        L.dspark_draft_sample_rnn.restype = ctypes.c_int
        L.dspark_draft_sample_rnn.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, u64,
                                              vp, vp, vp, vp, vp, vp, sz, vp]
        L.dspark_schedule_prefix.restype = ctypes.c_int
        L.dspark_schedule_prefix.argtypes = [vp, vp, vp, i32, i32, i32, i32, i32, vp, vp, vp, vp,
                                             vp, sz, vp]
        L.dspark_schedule_policy.restype = ctypes.c_int
        L.dspark_schedule_policy.argtypes = [vp, vp, vp, i32, i32, i32, i32, i32, i32, ctypes.c_float,
                                             vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
        L.dspark_verify.restype = ctypes.c_int
        L.dspark_verify.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                    i32, i32, i32, i32, i32, u64, vp, vp, vp, vp, vp, vp, sz, vp]
        L.dspark_verify_packed.restype = ctypes.c_int
        L.dspark_verify_packed.argtypes = [vp, vp, ctypes.c_int64] + L.dspark_verify.argtypes[1:]
        L.dspark_selftest_bounded_wait.restype = ctypes.c_int
        L.dspark_selftest_bounded_wait.argtypes = [ctypes.c_uint, ctypes.POINTER(ctypes.c_uint32), vp]
        L.dspark_pack_target.restype = ctypes.c_int
        L.dspark_pack_target.argtypes = [vp, vp, i32, i32, i32, i32, vp, vp, vp, vp]
        L.dspark_verify_noalloc.restype = ctypes.c_int
        L.dspark_verify_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                            i32, i32, i32, i32, i32, u64, vp, vp, vp, vp, vp, vp]
        L.dspark_read_device_flags.restype = ctypes.c_int
        L.dspark_read_device_flags.argtypes = [vp, vp, ctypes.POINTER(ctypes.c_uint32)]
        L.dspark_selftest_philox_rate.restype = ctypes.c_int
        L.dspark_selftest_philox_rate.argtypes = [vp, sz, i32, ctypes.POINTER(ctypes.c_double), vp]
        i64, cache_p = ctypes.c_int64, ctypes.POINTER(_CacheStruct)
        L.dspark_kv_append.restype = ctypes.c_int
        L.dspark_kv_append.argtypes = [cache_p, vp, vp, i64, i64, i32, vp, i32, vp, vp, i32, i32, vp]
        L.dspark_kv_read.restype = ctypes.c_int
        L.dspark_kv_read.argtypes = [cache_p, vp, i32, vp, vp, i32, i32, i32, vp, vp, vp]
        L.dspark_attention_workspace_bytes.restype = sz
        L.dspark_attention_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
        L.dspark_block_attention.restype = ctypes.c_int
        L.dspark_block_attention.argtypes = [cache_p, vp, i64, i32, i32, vp, i32, i32, vp, i32, vp, vp, i32, i32,
                                             i32, vp, ctypes.c_float, vp, vp, vp, sz, vp]
        L.dspark_window_workspace_bytes.restype = sz
        L.dspark_window_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
        L.dspark_window_attention.restype = ctypes.c_int
        L.dspark_window_attention.argtypes = [cache_p, vp, i64, i32, i32, vp, i32, i32, vp, i32, vp, vp, i32, i32, i32, i32,
                                              i32, vp, ctypes.c_float, vp, vp, vp, sz, vp]
        rotary_p = ctypes.POINTER(_RotaryStruct)
        L.dspark_rotary_rows.restype = ctypes.c_int
        L.dspark_rotary_rows.argtypes = [rotary_p, vp, i64, i64, i32, i32, i32, i32, vp, i32, vp, i64, i64, vp]
        L.dspark_kv_append_rotary.restype = ctypes.c_int
        L.dspark_kv_append_rotary.argtypes = [cache_p, rotary_p, vp, i64, i32, vp, vp, i64, i64, i32, vp, i32, vp, vp, i32,
                                              i32, vp, i64, vp, i64, vp]
        L.dspark_read_noalloc_flags.restype = ctypes.c_int
        L.dspark_read_noalloc_flags.argtypes = [vp, ctypes.POINTER(ctypes.c_uint32)]
        _lib = L
        return L


def _check(status):
    if status:
        raise DSparkError(status, load().dspark_last_error().decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _on_current_device(index, stream):
    """The library launches on the current device: a call's tensors, on device ``index``, and its stream have to be there."""
    if torch._C._cuda_getDevice() != index:
        raise ValueError("the tensors are on cuda:%d, which is not the current device" % index)
    if stream is not None and getattr(stream, "device_index", index) != index:
        raise ValueError("the stream is of cuda:%d, the tensors are on cuda:%d" % (stream.device_index, index))


def _stream(stream, device=None):
    if device is not None:
        _on_current_device(device.index, stream)
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


_AS_IT_IS = contextlib.nullcontext()


def _on(stream):
    """Where a call's own tensors are made: in the order of the stream that writes them (None: the current one).  Memory
    of another stream's order might still be read there, or be given away again before the call has run."""
    return _AS_IT_IS if stream is None else torch.cuda.stream(stream)


def _dtype_code(t):
    if t.dtype == torch.bfloat16:
        return DSPARK_BF16
    if t.dtype == torch.float32:
        return DSPARK_F32
    raise TypeError("logits must be bfloat16 or float32, got %s" % t.dtype)


def _need(t, name, dtype=None, shape=None, device=None):
    if t is None:
        raise ValueError("%s is required" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t


def _rid(request_id, B, device):
    if request_id is None:
        return None
    rid = request_id
    if rid.dtype not in (torch.int32,):
        raise TypeError("request_id must be int32 storage of uint32 ids")
    return _need(rid, "request_id", shape=(B,), device=device)


def version() -> int:
    return int(load().dspark_version())


def workspace_bytes(which: int, B: int, G: int, V: int, r: int) -> int:
    return int(load().dspark_workspace_bytes(which, B, G, V, r))


class WorkspaceCache:
    """Device scratch buffers reused across calls of the same shape."""

    def __init__(self):
        self._bufs = {}
        self._attention = {}
        self.lock = threading.Lock()    # held while a call that shares a buffer is enqueued

    def get(self, which, B, G, V, r, device):
        return self._sized(which, workspace_bytes(which, B, G, V, r), device)

    def attention(self, n, device, stream, raw):
        """An attention workspace of ``n`` bytes for a call on ``stream`` (None: the current one), whose handle is
        ``raw``: address, bytes and the tensor to hold until the call is enqueued.  One per stream, as calls on two
        streams may run at once; in a graph's capture one of the graph's own, which no later call can replace."""
        kept = self._attention.get((device, raw))
        with _on(stream):
            capturing = torch.cuda.is_current_stream_capturing()
        if capturing or kept is None or kept[1] < n:
            with _on(stream):
                buf = torch.empty(n + 256, dtype=torch.uint8, device=device)
            kept = (buf.data_ptr() + (-buf.data_ptr()) % 256, n, buf)
            if not capturing:
                self._attention[(device, raw)] = kept
        return kept

    def _sized(self, which, n, device):
        if n == 0:
            raise ValueError("invalid sizes for a workspace")
        key = (which, device)
        buf = self._bufs.get(key)
        if buf is None or buf.numel() < n:
            buf = torch.empty(n + 256, dtype=torch.uint8, device=device)
            self._bufs[key] = buf
        off = (-buf.data_ptr()) % 256
        return buf[off:off + n]


_default_ws = WorkspaceCache()


def draft_sample(base, e_in, w_out, anchor, temperature, request_id=None, seed=0, *,
                 out=None, store_logits=False, workspace=None, stream=None):
    """Draft one block per request.  Returns dict(tokens, lse, logq[, logits])."""
    lib = load()
    B, G, V = base.shape
    r = e_in.shape[1]
    dev = base.device
    _need(base, "base", shape=(B, G, V), device=dev)
    _need(e_in, "e_in", dtype=base.dtype, shape=(V, r), device=dev)
    _need(w_out, "w_out", dtype=base.dtype, shape=(V, r), device=dev)
    _need(anchor, "anchor", dtype=torch.int32, shape=(B,), device=dev)
    _need(temperature, "temperature", dtype=torch.float32, shape=(B,), device=dev)
    rid = _rid(request_id, B, dev)
    if out is None:
        with _on(stream):
            out = dict(tokens=torch.empty((B, G), dtype=torch.int32, device=dev),
                       lse=torch.empty((B, G), dtype=torch.float32, device=dev),
                       logq=torch.empty((B, G), dtype=torch.float32, device=dev))
            if store_logits:
                out["logits"] = torch.empty((B, G, V), dtype=torch.float32, device=dev)
    ws = workspace if workspace is not None else _default_ws.get(WS_DRAFT, B, G, V, r, dev)
    _check(lib.dspark_draft_sample(
        _ptr(base), _ptr(e_in), _ptr(w_out), _ptr(anchor), _ptr(temperature), _ptr(rid),
        B, G, V, r, _dtype_code(base), int(seed) & 0xFFFFFFFFFFFFFFFF,
        _ptr(out["tokens"]), _ptr(out["lse"]), _ptr(out["logq"]), _ptr(out.get("logits")),
        _ptr(ws), ws.numel(), _stream(stream, dev)))
    return out


def draft_sample_rnn(base, e_in, w_h, w_out, anchor, temperature, request_id=None, seed=0, *,
                     out=None, store_logits=False, store_states=False, workspace=None, stream=None):
    """Draft one block per request with the recurrent head (bf16 weights).

    Returns dict(tokens, lse, logq[, logits][, h]); ``h`` [B,G,r] bf16 are the
    states h_j.  Verify the block with :func:`verify` and ``draft_logits``."""
    lib = load()
    B, G, V = base.shape
    r = e_in.shape[1]
    dev = base.device
    _need(base, "base", dtype=torch.bfloat16, shape=(B, G, V), device=dev)
    _need(e_in, "e_in", dtype=torch.bfloat16, shape=(V, r), device=dev)
    _need(w_h, "w_h", dtype=torch.bfloat16, shape=(r, r), device=dev)
    _need(w_out, "w_out", dtype=torch.bfloat16, shape=(V, r), device=dev)
    _need(anchor, "anchor", dtype=torch.int32, shape=(B,), device=dev)
    _need(temperature, "temperature", dtype=torch.float32, shape=(B,), device=dev)
    rid = _rid(request_id, B, dev)
    if out is None:
        with _on(stream):
            out = dict(tokens=torch.empty((B, G), dtype=torch.int32, device=dev),
                       lse=torch.empty((B, G), dtype=torch.float32, device=dev),
                       logq=torch.empty((B, G), dtype=torch.float32, device=dev))
            if store_logits:
                out["logits"] = torch.empty((B, G, V), dtype=torch.float32, device=dev)
            if store_states:
                out["h"] = torch.empty((B, G, r), dtype=torch.bfloat16, device=dev)
    ws = workspace if workspace is not None else _default_ws.get(WS_DRAFT_RNN, B, G, V, r, dev)
    _check(lib.dspark_draft_sample_rnn(
        _ptr(base), _ptr(e_in), _ptr(w_h), _ptr(w_out), _ptr(anchor), _ptr(temperature), _ptr(rid),
        B, G, V, r, DSPARK_BF16, int(seed) & 0xFFFFFFFFFFFFFFFF,
        _ptr(out["tokens"]), _ptr(out["lse"]), _ptr(out["logq"]), _ptr(out.get("logits")),
        _ptr(out.get("h")), _ptr(ws), ws.numel(), _stream(stream, dev)))
    return out


# verify-length policies of dspark_schedule_policy
SCHED_EARLY_STOP, SCHED_BEST_PREFIX, SCHED_THRESHOLD_CUM, SCHED_THRESHOLD_CONF = 0, 1, 2, 3


def schedule_prefix(conf_logits, pos_temp, sps, L_min, L_max, *, policy=SCHED_EARLY_STOP, threshold=0.0,
                    out=None, workspace=None, stream=None):
    """Calibrate confidences and choose verify lengths (early stop by default;
    ``policy`` selects another rule of dspark_schedule_policy).

    Returns dict(conf, cum_conf, verify_len, theta)."""
    lib = load()
    B, G = conf_logits.shape
    dev = conf_logits.device
    _need(conf_logits, "conf_logits", dtype=torch.float32, device=dev)
    _need(pos_temp, "pos_temp", dtype=torch.float32, shape=(G,), device=dev)
    _need(sps, "sps", dtype=torch.float32, device=dev)
    if out is None:
        with _on(stream):
            out = dict(conf=torch.empty((B, G), dtype=torch.float32, device=dev),
                       cum_conf=torch.empty((B, G), dtype=torch.float32, device=dev),
                       verify_len=torch.empty((B,), dtype=torch.int32, device=dev),
                       theta=torch.empty((1,), dtype=torch.float64, device=dev))
    ws = workspace if workspace is not None else _default_ws.get(WS_SCHEDULE, B, G, 8, 1, dev)
    _check(lib.dspark_schedule_policy(
        _ptr(conf_logits), _ptr(pos_temp), _ptr(sps), sps.numel(), B, G, int(L_min), int(L_max),
        int(policy), float(threshold),
        _ptr(out["conf"]), _ptr(out["cum_conf"]), _ptr(out["verify_len"]), _ptr(out.get("theta")),
        _ptr(ws), ws.numel(), _stream(stream, dev)))
    return out


class LaggedScheduler:
    """The deployed scheduling mode: round t's verify lengths come from the
    calibrated confidences of round t - ``lag`` ("DSpark, la bozza che sa quando
    fermarsi", section "Che cosa resta da verificare": the production scheduler
    works from confidences two rounds old and has no early stop), so the
    schedule need not wait for the current round's confidence head.

    Keeps a device ring of the last ``lag`` rounds' confidence logits [B, G];
    until it has filled, a round is scheduled from its own logits.  Each
    :meth:`step` runs one dspark_schedule_policy launch (policy ``policy``,
    best prefix by default) and returns its outputs."""

    def __init__(self, pos_temp, sps, L_min, L_max, *, lag=2, policy=SCHED_BEST_PREFIX, threshold=0.0):
        if lag < 0:
            raise ValueError("lag must be >= 0")
        self.pos_temp, self.sps = pos_temp, sps
        self.L_min, self.L_max = int(L_min), int(L_max)
        self.lag, self.policy, self.threshold = int(lag), int(policy), float(threshold)
        self._ring = []

    def step(self, conf_logits, *, out=None, stream=None):
        """Schedule this round; ``conf_logits`` [B, G] are this round's logits."""
        src = self._ring[0] if len(self._ring) == self.lag and self.lag > 0 else conf_logits
        res = schedule_prefix(src, self.pos_temp, self.sps, self.L_min, self.L_max, policy=self.policy,
                              threshold=self.threshold, out=out, stream=stream)
        if self.lag > 0:
            with _on(stream):
                self._ring.append(conf_logits.clone())
            if len(self._ring) > self.lag:
                self._ring.pop(0)
        return res


def verify(target, base, e_in, w_out, anchor, draft, verify_len, temperature, request_id=None,
           seed=0, *, draft_logits=None, target_row0=None, out=None, workspace=None, stream=None):
    """Verify one drafted block per request.

    ``draft`` is the dict returned by :func:`draft_sample`.  ``target`` is
    [B, G+1, V], or with ``target_row0`` ([B] int64) the packed rows [n, V]
    (request b's row j at row target_row0[b] + j, see dspark_verify_packed).
    Returns dict(accept_len, out_tokens, num_out, target_lse, logp)."""
    lib = load()
    B, G = draft["tokens"].shape
    V = target.shape[-1]
    dev = target.device
    if target_row0 is None:
        _need(target, "target", shape=(B, G + 1, V), device=dev)
    else:
        _need(target, "target", device=dev)
        if target.dim() != 2:
            raise ValueError("a packed target is [rows, V]")
        _need(target_row0, "target_row0", dtype=torch.int64, shape=(B,), device=dev)
    if draft_logits is None:
        _need(base, "base", dtype=target.dtype, shape=(B, G, V), device=dev)
        _need(e_in, "e_in", dtype=target.dtype, device=dev)
        _need(w_out, "w_out", dtype=target.dtype, device=dev)
        r = e_in.shape[1]
    else:
        _need(draft_logits, "draft_logits", dtype=torch.float32, shape=(B, G, V), device=dev)
        r = e_in.shape[1] if e_in is not None else 16
    _need(anchor, "anchor", dtype=torch.int32, shape=(B,), device=dev)
    for k in ("tokens", "lse", "logq"):
        _need(draft[k], "draft." + k, shape=(B, G), device=dev)
    if verify_len is not None:
        _need(verify_len, "verify_len", dtype=torch.int32, shape=(B,), device=dev)
    _need(temperature, "temperature", dtype=torch.float32, shape=(B,), device=dev)
    rid = _rid(request_id, B, dev)
    if out is None:
        with _on(stream):
            out = dict(accept_len=torch.empty((B,), dtype=torch.int32, device=dev),
                       out_tokens=torch.empty((B, G + 1), dtype=torch.int32, device=dev),
                       num_out=torch.empty((B,), dtype=torch.int32, device=dev),
                       target_lse=torch.empty((B, G + 1), dtype=torch.float32, device=dev),
                       logp=torch.empty((B, G), dtype=torch.float32, device=dev))
    ws = workspace if workspace is not None else _default_ws.get(WS_VERIFY, B, G, V, r, dev)
    args = (_ptr(base), _ptr(e_in), _ptr(w_out), _ptr(draft_logits), _ptr(anchor),
            _ptr(draft["tokens"]), _ptr(draft["lse"]), _ptr(draft["logq"]), _ptr(verify_len),
            _ptr(temperature), _ptr(rid), B, G, V, r, _dtype_code(target),
            int(seed) & 0xFFFFFFFFFFFFFFFF,
            _ptr(out["accept_len"]), _ptr(out["out_tokens"]), _ptr(out["num_out"]),
            _ptr(out.get("target_lse")), _ptr(out.get("logp")), _ptr(ws), ws.numel(),
            _stream(stream, dev))
    if target_row0 is None:
        _check(lib.dspark_verify(_ptr(target), *args))
    else:
        _check(lib.dspark_verify_packed(_ptr(target), _ptr(target_row0), target.shape[0], *args))
    return out


def pack_target(target, verify_len, *, out=None, stream=None):
    """Rows 0 .. L_b of every request of ``target`` [B, G+1, V] (device, or
    pinned host memory, which the device reads directly) packed for
    :func:`verify` with ``target_row0`` (dspark_pack_target).

    Returns dict(target [B*(G+1), V] with the packed rows first, row0 [B]
    int64, n_rows [1] int64), all on the device of ``verify_len``."""
    lib = load()
    B, G1, V = target.shape
    dev = verify_len.device if verify_len is not None else torch.device("cuda", torch.cuda.current_device())
    if not target.is_contiguous():
        raise ValueError("target must be contiguous")
    if target.device.type == "cpu" and not target.is_pinned():
        raise ValueError("a host target must be in pinned memory")
    if verify_len is not None:
        _need(verify_len, "verify_len", dtype=torch.int32, shape=(B,), device=dev)
    if out is None:
        with _on(stream):
            out = dict(target=torch.empty((B * G1, V), dtype=target.dtype, device=dev),
                       row0=torch.empty((B,), dtype=torch.int64, device=dev),
                       n_rows=torch.empty((1,), dtype=torch.int64, device=dev))
    _check(lib.dspark_pack_target(_ptr(target), _ptr(verify_len), B, G1 - 1, V, _dtype_code(target),
                                  _ptr(out["target"]), _ptr(out["row0"]), _ptr(out.get("n_rows")),
                                  _stream(stream, dev)))
    return out


# ------------------------------------------------- quantised cache, attention
_KV_FORMATS = {torch.float8_e4m3fn: KV_E4M3, torch.int8: KV_INT8}
_ROW_DTYPES = {torch.bfloat16: DSPARK_BF16, torch.float32: DSPARK_F32, torch.float16: DSPARK_F16}
_MASKS = {"causal": MASK_CAUSAL, "full": MASK_FULL}


class KVCache:
    """A paged, quantised key/value cache (struct dspark_kv_cache).

    ``k`` and ``v`` [n_pages, n_kv_heads, page_size, head_dim] hold float8_e4m3fn
    or int8 codes, ``k_scale`` and ``v_scale`` [n_pages, n_kv_heads, page_size]
    fp32 one scale per token and head.  ``flags`` is the device flag word that
    the calls on this cache OR their bits into: read it with
    :func:`read_device_flags`, clear it with ``cache.flags.zero_()``."""

    def __init__(self, k, v, k_scale, v_scale):
        if k.dtype not in _KV_FORMATS:
            raise TypeError("cache codes must be float8_e4m3fn or int8, got %s" % k.dtype)
        if k.dim() != 4:
            raise ValueError("cache codes are [n_pages, n_kv_heads, page_size, head_dim]")
        _need(k, "k")
        _need(v, "v", dtype=k.dtype, shape=k.shape, device=k.device)
        _need(k_scale, "k_scale", dtype=torch.float32, shape=k.shape[:3], device=k.device)
        _need(v_scale, "v_scale", dtype=torch.float32, shape=k.shape[:3], device=k.device)
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.flags = torch.zeros(64, dtype=torch.int32, device=k.device)
        self.n_pages, self.n_kv_heads, self.page_size, self.head_dim = k.shape
        self.device = k.device
        self._index = k.get_device()
        self.struct = _CacheStruct(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                                   self.flags.data_ptr(), *k.shape, _KV_FORMATS[k.dtype])
        self._ref = ctypes.byref(self.struct)

    @classmethod
    def empty(cls, n_pages, n_kv_heads, page_size, head_dim, *, dtype=torch.float8_e4m3fn, device="cuda"):
        """A cache of zero codes and zero scales."""
        shape = (n_pages, n_kv_heads, page_size, head_dim)
        codes = [torch.zeros(shape, dtype=torch.uint8, device=device).view(dtype) for _ in range(2)]
        return cls(*codes, *[torch.zeros(shape[:3], dtype=torch.float32, device=device) for _ in range(2)])


# These calls take some ten microseconds on the device, so their checks are made in one expression each;
# only a failed one is looked at again for its message.
def _vec(t, name, dtype, n, cache):
    if t.dtype is dtype and t.dim() == 1 and t.shape[0] == n and t.get_device() == cache._index and t.is_contiguous():
        return t.data_ptr()
    _need(t, name, dtype=dtype, shape=(n,), device=cache.device)
    raise ValueError("%s must be on %s" % (name, cache.device))


def _row_stride(t, name, heads, cache):
    """Checks packed rows [n, heads, D], whose rows may lie any 16-byte multiple
    apart; returns their distance in elements."""
    n, h, d = t.shape
    if t.get_device() != cache._index:
        raise ValueError("%s must be on %s" % (name, cache.device))
    if h != heads or d != cache.head_dim:
        raise ValueError("%s must have shape (rows, %d, %d), got %s" % (name, heads, cache.head_dim, tuple(t.shape)))
    row, head, elem = t.stride()
    if elem != 1 or (h > 1 and head != d):
        raise ValueError("the heads of a row of %s must be contiguous" % name)
    return row if n > 1 else h * d


def _paged(block_table, start, name, row0, cache, n_rows, n_tokens=0, n_pages=0):
    B, max_pages = block_table.shape
    # ctypes would pass on the low 32 bits of a larger number (one below 0 the library refuses)
    if (n_rows | n_tokens | n_pages | B | max_pages) >> 31:
        if any(not -0x80000000 <= n <= 0x7fffffff for n in (n_rows, n_tokens, n_pages, B, max_pages)):
            raise ValueError("numbers of requests, pages, rows and tokens must be below 2^31")
    if not (block_table.dtype is torch.int32 and block_table.get_device() == cache._index and block_table.is_contiguous()):
        _need(block_table, "block_table", dtype=torch.int32, device=cache.device)
    return (B, max_pages, block_table.data_ptr(), _vec(start, name, torch.int32, B, cache),
            _vec(row0, "row0", torch.int64, B + 1, cache))


def _raw_stream(stream, cache):
    if stream is None and torch._C._cuda_getDevice() == cache._index:
        return torch._C._cuda_getCurrentRawStream(cache._index)
    _on_current_device(cache._index, stream)
    return stream.cuda_stream


def kv_append(k, v, cache, block_table, start, row0, *, stream=None):
    """Quantise packed rows ``k``, ``v`` [n_rows, n_kv_heads, head_dim] into
    ``cache``: row i of request b (rows row0[b] .. row0[b+1] - 1, ``row0``
    [B+1] int64) at position start[b] + i of the request's pages
    (``block_table`` [B, max_pages] int32).  See dspark_kv_append."""
    lib = _lib or load()
    raw = _raw_stream(stream, cache)
    shape, dtype = k.shape, k.dtype
    n = shape[0]
    B, max_pages, table_p, start_p, row0_p = _paged(block_table, start, "start", row0, cache, n)
    code = _ROW_DTYPES.get(dtype)
    if code is None or v.dtype is not dtype or v.shape != shape:
        raise TypeError("k and v must have one shape and one of the types bf16, fp16 and fp32")
    ks = _row_stride(k, "k", cache.n_kv_heads, cache)
    vs = _row_stride(v, "v", cache.n_kv_heads, cache)
    _check(lib.dspark_kv_append(cache._ref, k.data_ptr(), v.data_ptr(), ks, vs, code, row0_p, n, start_p, table_p,
                                max_pages, B, raw))


# 2 ** 64 turns' parts a radian: 2 ** 64 / (2 pi)
_PARTS_PER_RADIAN = Fraction(2 ** 64, 2) / Fraction("3.14159265358979323846264338327950288419716939937510582097494459")


class Rotary:
    """Frequencies of rotary positions (struct dspark_rotary).

    ``inv_freq`` (numbers or a 1-D tensor, taken as they are in 64 bits) is the
    angle in radians that a step of one position adds to each pair.  Pair i of a
    head of D elements is elements i and n + i of its first 2 n (n = len(inv_freq),
    a multiple of 4, 2 n <= D), or with ``adjacent`` 2 i and 2 i + 1; the others pass
    as they are.  ``axis`` names the axis of positions (0, 1, ..) that turns each
    pair, for positions of several axes (time, height, width)."""

    def __init__(self, inv_freq, *, axis=None, adjacent=False, device="cuda"):
        freq = [float(w) for w in (inv_freq.tolist() if isinstance(inv_freq, torch.Tensor) else inv_freq)]
        if not all(math.isfinite(w) for w in freq):
            raise ValueError("inv_freq must be finite")
        self.n_pairs, self.n_axes, self.adjacent = len(freq), 1, bool(adjacent)
        if self.n_pairs < 4 or self.n_pairs % 4:
            raise ValueError("the number of frequencies must be a positive multiple of 4, got %d" % self.n_pairs)
        steps = [round(Fraction(w) * _PARTS_PER_RADIAN) % 2 ** 64 for w in freq]
        self.step = torch.tensor([t - 2 ** 64 if t >> 63 else t for t in steps], dtype=torch.int64).to(device)
        self.axis = None
        if axis is not None:
            axis = [int(i) for i in axis]
            if len(axis) != self.n_pairs or min(axis) < 0 or max(axis) >= 16:
                raise ValueError("axis must name an axis in [0, 16) for each of the %d pairs" % self.n_pairs)
            self.n_axes = max(axis) + 1
            self.axis = torch.tensor(axis, dtype=torch.int32).to(device)
        self.device = self.step.device
        self._index = self.step.get_device()
        self.struct = _RotaryStruct(self.step.data_ptr(), None if self.axis is None else self.axis.data_ptr(), self.n_pairs,
                                    self.n_axes, int(self.adjacent))
        self._ref = ctypes.byref(self.struct)


def _positions(t, rotary, n):
    """Address of positions [n_axes, n] int32 (or [n] of one axis)."""
    if not (t.dtype is torch.int32 and t.get_device() == rotary._index and t.is_contiguous() and t.numel() == rotary.n_axes * n
            and (t.dim() == 2 and t.shape[0] == rotary.n_axes or t.dim() == 1 and rotary.n_axes == 1)):
        _need(t, "positions", dtype=torch.int32, shape=(rotary.n_axes, n), device=rotary.device)
    return t.data_ptr()


def rotary(x, rotary, positions, *, inverse=False, out=None, stream=None):
    """Rows ``x`` [n_rows, heads, head_dim] turned by their ``positions``
    ([n_axes, n_rows] int32, or [n_rows] of one axis), or turned back with
    ``inverse``, which is also the turning's gradient.  The rows and the heads of
    ``x`` may lie apart by strides of 16-byte multiples (slices of a fused
    projection, or a transposed heads-first tensor); ``out`` may be ``x``.
    Returns the turned rows, in the layout of ``x`` when that has no gaps.  See
    dspark_rotary_rows."""
    lib = _lib or load()
    raw = _raw_stream(stream, rotary)
    n, heads, d = x.shape
    code = _ROW_DTYPES.get(x.dtype)
    if code is None:
        raise TypeError("rows must be bf16, fp16 or fp32, got %s" % x.dtype)
    positions_p = _positions(positions, rotary, n)
    if out is None:
        with _on(stream):
            out = torch.empty_like(x)
    elif out.dtype is not x.dtype or out.shape != x.shape:
        raise ValueError("out must have the shape and type of x")
    row, head, elem = x.stride()
    out_row, out_head, out_elem = out.stride()
    if x.get_device() != rotary._index or out.get_device() != rotary._index:
        raise ValueError("x and out must be on %s" % rotary.device)
    if (elem != 1 or out_elem != 1) and d > 1:
        raise ValueError("the elements of a head of x and out must be contiguous")
    if (n | heads | d) >> 31:
        raise ValueError("numbers of rows and heads must be below 2^31")
    _check(lib.dspark_rotary_rows(rotary._ref, x.data_ptr(), row, head, n, heads, d, code, positions_p, int(bool(inverse)),
                                  out.data_ptr(), out_row, out_head, raw))
    return out


def kv_append_rotary(k, v, cache, block_table, start, row0, rotary, *, q=None, positions=None, offset=0, out=None,
                     stream=None):
    """:func:`kv_append` with the keys turned by their positions on the way, and
    the queries ``q`` [n_rows, n_q_heads, head_dim] of the same rows turned beside
    them, to ``out`` (made here by default; ``q`` itself turns them in place).  Row i
    of request b is at position ``offset`` + start[b] + i on every axis, or where
    ``positions`` ([n_axes, n_rows] int32, or [n_rows] of one axis) says.  See
    dspark_kv_append_rotary.

    Returns the turned queries, None without ``q``; rows of no request stay as
    they were in ``out``."""
    lib = _lib or load()
    raw = _raw_stream(stream, cache)
    shape, dtype = k.shape, k.dtype
    n = shape[0]
    B, max_pages, table_p, start_p, row0_p = _paged(block_table, start, "start", row0, cache, n)
    code = _ROW_DTYPES.get(dtype)
    if code is None or v.dtype is not dtype or v.shape != shape:
        raise TypeError("k and v must have one shape and one of the types bf16, fp16 and fp32")
    if rotary._index != cache._index:
        raise ValueError("rotary must be on %s" % cache.device)
    ks = _row_stride(k, "k", cache.n_kv_heads, cache)
    vs = _row_stride(v, "v", cache.n_kv_heads, cache)
    positions_p = None if positions is None else _positions(positions, rotary, n)
    offset = int(offset)
    if not -2 ** 62 <= offset <= 2 ** 62:
        raise ValueError("offset is out of range")
    q_p = out_p = None
    qs = outs = heads = 0
    if q is not None:
        heads = q.shape[1]
        if q.dtype is not dtype or q.shape[0] != n:
            raise TypeError("q must have the type and the rows of k")
        qs = _row_stride(q, "q", heads, cache)
        if out is None:
            with _on(stream):
                out = torch.empty(q.shape, dtype=dtype, device=cache.device)
        elif out.dtype is not dtype or out.shape != q.shape:
            raise ValueError("out must have the shape and type of q")
        outs = _row_stride(out, "out", heads, cache)
        q_p, out_p = q.data_ptr(), out.data_ptr()
    elif out is not None:
        raise ValueError("out is for turned queries: q is required")
    _check(lib.dspark_kv_append_rotary(cache._ref, rotary._ref, q_p, qs, heads, k.data_ptr(), v.data_ptr(), ks, vs, code,
                                       row0_p, n, start_p, table_p, max_pages, B, positions_p, offset, out_p, outs, raw))
    return out


def kv_read(cache, block_table, start, row0, n_rows, *, dtype=torch.bfloat16, out=None, stream=None):
    """Cached tokens as packed rows: row i of request b is position
    start[b] + i.  Returns dict(k, v) of [n_rows, n_kv_heads, head_dim]; an
    ``out`` with only one of them reads that one.  See dspark_kv_read."""
    lib = _lib or load()
    dev = cache.device
    raw = _raw_stream(stream, cache)
    B, max_pages, table_p, start_p, row0_p = _paged(block_table, start, "start", row0, cache, n_rows)
    if dtype not in _ROW_DTYPES:
        raise TypeError("rows must be bf16, fp16 or fp32, got %s" % dtype)
    shape = (n_rows, cache.n_kv_heads, cache.head_dim)
    if out is None:
        with _on(stream):
            out = dict(k=torch.empty(shape, dtype=dtype, device=dev), v=torch.empty(shape, dtype=dtype, device=dev))
    else:
        for name in out:
            _need(out[name], name, dtype=dtype, shape=shape, device=dev)
    _check(lib.dspark_kv_read(cache._ref, row0_p, n_rows, start_p, table_p, max_pages, B, _ROW_DTYPES[dtype],
                              _ptr(out.get("k")), _ptr(out.get("v")), raw))
    return out


@functools.lru_cache(maxsize=1024)
def attention_workspace_bytes(B, n_rows, n_q_heads, n_kv_heads, head_dim) -> int:
    return int(load().dspark_attention_workspace_bytes(B, n_rows, n_q_heads, n_kv_heads, head_dim))


def block_attention(q, cache, block_table, kv_len, row0, *, prefix_pages=None, prefix_len=0, mask="causal",
                    row_mask=None, scale=None, out=None, workspace=None, stream=None):
    """Attention of every request's block rows ``q`` [n_rows, n_q_heads,
    head_dim] (row i of request b is row row0[b] + i) over the first
    ``prefix_len`` tokens of ``prefix_pages`` (int32), which all requests share,
    and over the request's own kv_len[b] cached tokens, the last ones of which
    are the block itself.  ``mask`` ("causal" or "full") or ``row_mask``
    ([n_rows] int64, bit t: the row sees token t of its block) rules inside the
    block; ``scale`` is head_dim ** -0.5 by default.  Without a ``workspace``
    (attention_workspace_bytes, 256-byte aligned) one is kept per stream.  See dspark_block_attention.

    Returns dict(out, lse): out like q, lse [n_rows, n_q_heads] fp32."""
    return _attention(None, q, cache, block_table, kv_len, row0, prefix_pages, prefix_len, mask, row_mask, scale, out,
                      workspace, stream)


@functools.lru_cache(maxsize=1024)
def window_workspace_bytes(B, n_rows, n_q_heads, n_kv_heads, head_dim) -> int:
    return int(load().dspark_window_workspace_bytes(B, n_rows, n_q_heads, n_kv_heads, head_dim))


def window_attention(q, cache, block_table, kv_len, row0, *, window, sinks=0, prefix_pages=None, prefix_len=0,
                     mask="causal", row_mask=None, scale=None, out=None, workspace=None, stream=None):
    """:func:`block_attention` through a window: a row sees the last ``window``
    tokens up to its own and the first ``sinks`` ones (of the prefix, then of the
    request's own), as far as ``mask`` or ``row_mask`` shows them to it; a row with a
    mask word stands behind the word's tokens (``window`` is at least 64 then).
    Pages before the block that neither reaches are not read.  See
    dspark_window_attention.

    Returns dict(out, lse): out like q, lse [n_rows, n_q_heads] fp32."""
    window, sinks = int(window), int(sinks)
    if window > 0x7fffffff or sinks > 0x7fffffff or window < 0 or sinks < 0:
        # (more than any cache holds is all of it; what is below 0 the library refuses)
        window, sinks = (max(-1, min(x, 0x7fffffff)) for x in (window, sinks))
    return _attention((window, sinks), q, cache, block_table, kv_len, row0, prefix_pages, prefix_len, mask,
                      row_mask, scale, out, workspace, stream)


def _attention(window, q, cache, block_table, kv_len, row0, prefix_pages, prefix_len, mask, row_mask, scale, out, workspace,
               stream):
    """block_attention, or with (window, sinks) window_attention"""
    lib = _lib or load()
    dev = cache.device
    raw = _raw_stream(stream, cache)
    prefix_len = int(prefix_len)
    n_pages = 0 if prefix_pages is None else prefix_pages.numel()
    B, max_pages, table_p, len_p, row0_p = _paged(block_table, kv_len, "kv_len", row0, cache, q.shape[0], prefix_len, n_pages)
    if q.dtype is not torch.bfloat16 and q.dtype is not torch.float16:
        raise TypeError("q must be bfloat16 or float16, got %s" % q.dtype)
    n, Hq, D = q.shape
    qs = _row_stride(q, "q", Hq, cache)
    pages_p = None if prefix_pages is None else _vec(prefix_pages, "prefix_pages", torch.int32, n_pages, cache)
    words_p = None if row_mask is None else _vec(row_mask, "row_mask", torch.int64, n, cache)
    if out is None:
        with _on(stream):
            out = dict(out=torch.empty((n, Hq, D), dtype=q.dtype, device=dev),
                       lse=torch.empty((n, Hq), dtype=torch.float32, device=dev))
        lse_p = out["lse"].data_ptr()
    else:
        _need(out["out"], "out", dtype=q.dtype, shape=(n, Hq, D), device=dev)
        lse_p = None
        if out.get("lse") is not None:
            _need(out["lse"], "lse", dtype=torch.float32, shape=(n, Hq), device=dev)
            lse_p = out["lse"].data_ptr()
    scale = D ** -0.5 if scale is None else float(scale)
    if window is not None and workspace is None and not window_workspace_bytes(B, n, Hq, cache.n_kv_heads, D):
        _check(lib.dspark_window_attention(
            cache._ref, q.data_ptr(), qs, _ROW_DTYPES[q.dtype], Hq, row0_p, n, B, table_p, max_pages, len_p, pages_p, n_pages,
            prefix_len, window[0], window[1], _MASKS[mask], words_p, scale, out["out"].data_ptr(), lse_p, None, 0, raw))
        return out
    # (two launches that meet in the workspace: another thread's must not come in between)
    with _default_ws.lock if workspace is None else _AS_IT_IS:
        if workspace is None:
            size = attention_workspace_bytes if window is None else window_workspace_bytes
            ws_p, ws_n, workspace = _default_ws.attention(size(B, n, Hq, cache.n_kv_heads, D), dev, stream, raw)
        else:
            _need(workspace, "workspace", device=dev)
            ws_p, ws_n = workspace.data_ptr(), workspace.numel()
        if window is None:
            status = lib.dspark_block_attention(
                cache._ref, q.data_ptr(), qs, _ROW_DTYPES[q.dtype], Hq, row0_p, n, B, table_p, max_pages, len_p, pages_p,
                n_pages, prefix_len, _MASKS[mask], words_p, scale, out["out"].data_ptr(), lse_p, ws_p, ws_n, raw)
        else:
            status = lib.dspark_window_attention(
                cache._ref, q.data_ptr(), qs, _ROW_DTYPES[q.dtype], Hq, row0_p, n, B, table_p, max_pages, len_p, pages_p,
                n_pages, prefix_len, window[0], window[1], _MASKS[mask], words_p, scale, out["out"].data_ptr(), lse_p, ws_p,
                ws_n, raw)
    _check(status)
    return out


NOALLOC_SCRATCH_BYTES = 4 << 20


def verify_noalloc(target, base, e_in, w_out, anchor, draft, verify_len, temperature,
                   request_id=None, seed=0, *, draft_logits=None, out=None, stream=None):
    """:func:`verify` through ``dspark_verify_noalloc``: no workspace is passed
    or allocated; the library uses its fixed device scratch array."""
    lib = load()
    B, G1, V = target.shape
    G = G1 - 1
    dev = target.device
    _need(target, "target", device=dev)
    r = e_in.shape[1] if e_in is not None else 16
    if out is None:
        with _on(stream):
            out = dict(accept_len=torch.empty((B,), dtype=torch.int32, device=dev),
                       out_tokens=torch.empty((B, G + 1), dtype=torch.int32, device=dev),
                       num_out=torch.empty((B,), dtype=torch.int32, device=dev),
                       target_lse=torch.empty((B, G + 1), dtype=torch.float32, device=dev),
                       logp=torch.empty((B, G), dtype=torch.float32, device=dev))
    rid = _rid(request_id, B, dev)
    _check(lib.dspark_verify_noalloc(
        _ptr(target), _ptr(base), _ptr(e_in), _ptr(w_out), _ptr(draft_logits), _ptr(anchor),
        _ptr(draft["tokens"]), _ptr(draft["lse"]), _ptr(draft["logq"]), _ptr(verify_len),
        _ptr(temperature), _ptr(rid), B, G, V, r, _dtype_code(target),
        int(seed) & 0xFFFFFFFFFFFFFFFF,
        _ptr(out["accept_len"]), _ptr(out["out_tokens"]), _ptr(out["num_out"]),
        _ptr(out.get("target_lse")), _ptr(out.get("logp")), _stream(stream, dev)))
    return out


def selftest_bounded_wait(limit_us=1000, stream=None) -> int:
    """Run dspark_selftest_bounded_wait: 3 when both probe waits report their
    timeout."""
    val = ctypes.c_uint32(0)
    _check(load().dspark_selftest_bounded_wait(int(limit_us), ctypes.byref(val), _stream(stream)))
    return int(val.value)


def selftest_philox_rate(iters=2048, stream=None) -> float:
    """Philox4x32-10 blocks per second of the draft's word code on this
    device (dspark_selftest_philox_rate)."""
    dev = torch.device("cuda", torch.cuda.current_device())
    sink = torch.empty(1 << 16, dtype=torch.uint8, device=dev)
    val = ctypes.c_double(0.0)
    _check(load().dspark_selftest_philox_rate(_ptr(sink), sink.numel(), int(iters), ctypes.byref(val),
                                              _stream(stream)))
    return float(val.value)


def read_device_flags(workspace, stream=None) -> int:
    val = ctypes.c_uint32(0)
    _check(load().dspark_read_device_flags(_ptr(workspace), _stream(stream), ctypes.byref(val)))
    return int(val.value)


def read_noalloc_flags(stream=None) -> int:
    """The flag word of the last :func:`verify_noalloc` call."""
    val = ctypes.c_uint32(0)
    _check(load().dspark_read_noalloc_flags(_stream(stream), ctypes.byref(val)))
    return int(val.value)


def default_workspace(which, B, G, V, r, device):
    return _default_ws.get(which, B, G, V, r, device)
