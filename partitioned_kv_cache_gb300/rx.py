"""Python binding of librx.so (the C ABI in include/rx.h).

Argument marshalling only: every step of the hot path runs in the library's
CUDA kernels.  PyTorch supplies device memory and the current stream.  Import
fails loudly when the library has not been built -- there is no fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import List, NamedTuple, Optional, Sequence, Tuple

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "librx.so")
if not os.path.exists(_LIB_PATH):
    raise ImportError(
        "librx.so is not built (expected at %s); run `python -c \"import __graft_entry__ as g; "
        "g.build()\"` or `python -m partitioned_kv_cache_gb300.build`" % _LIB_PATH)
_lib = ctypes.CDLL(_LIB_PATH)

RX_OK = 0
STATUS_NAMES = {0: "RX_OK", -1: "RX_ERR_ARG", -2: "RX_ERR_LAYER", -3: "RX_ERR_CAPACITY",
                -4: "RX_ERR_CUDA", -5: "RX_ERR_TIMEOUT", -6: "RX_ERR_UNSUPPORTED",
                -7: "RX_ERR_STATE"}

#: Every symbol include/rx.h declares.
EXPORTS = ("rx_cache_create", "rx_cache_destroy", "rx_pin_prefix", "rx_push_frame",
           "rx_attend_suffix", "rx_attend_batch", "rx_ada_gamma", "rx_adarmsnorm",
           "rx_get_state", "rx_debug_window", "rx_export_window", "rx_check_device_error",
           "rx_set_attn_splits", "rx_launch_count", "rx_status_str", "rx_last_error",
           "rx_attend_regions_static", "rx_attend_suffix_block_causal", "rx_tail_append",
           "rx_snapshot_bytes", "rx_snapshot", "rx_restore", "rx_push_frame_async",
           "rx_set_attn_dparts", "rx_debug_inject_timeout", "rx_debug_choose_partition",
           "rx_attend_suffix_norms", "rx_attend_batch_norms", "rx_tail_append_quant",
           "rx_attend_streams_quant", "rx_verify_drafts", "rx_debug_choose_stream_partition",
           "rx_rotate_heads", "rx_rotate_heads_paged", "rx_attend_pages", "rx_attend_pages_workspace",
           "rx_weigh_pages", "rx_weigh_pages_workspace", "rx_evict_pages", "rx_debug_page_plan")


class RxConfig(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in
                ("L", "Hq", "Hkv", "D", "P_cap", "N", "F", "S_cap", "tail_cap", "max_req",
                 "spare_slot")]


class RxStreamBatch(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k_tail", ctypes.c_void_p), ("v_tail", ctypes.c_void_p),
                ("tail_len", ctypes.c_void_p), ("out", ctypes.c_void_p), ("B", ctypes.c_int),
                ("T", ctypes.c_int)]


class RxQuantStreams(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("q", "k_tail", "v_tail", "k_exp", "v_exp", "tail_len", "n_new", "out")] + \
               [("B", ctypes.c_int), ("T", ctypes.c_int)]


class RxNormRows(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("gamma", ctypes.c_void_p), ("y", ctypes.c_void_p),
                ("rows", ctypes.c_int), ("d", ctypes.c_int), ("eps", ctypes.c_float)]


MAX_AXES = 4


class RxPages(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "weight", "table")] + \
               [(n, ctypes.c_int) for n in ("n_pages", "page", "max_pages", "B")]


class RxHeads(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("freq", "q_weight", "k_weight")] + \
               [(n, ctypes.c_int) for n in ("Hq", "Hkv", "D", "n_axes")] + \
               [("sections", ctypes.c_int * MAX_AXES), ("adjacent", ctypes.c_int), ("eps", ctypes.c_float)]


MAX_NORM_JOBS = 2

_vp, _i, _f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
_sigs = {
    "rx_cache_create": (_i, [ctypes.POINTER(RxConfig), ctypes.POINTER(_vp)]),
    "rx_cache_destroy": (_i, [_vp]),
    "rx_pin_prefix": (_i, [_vp, _vp, _vp, _i, _vp]),
    "rx_push_frame": (_i, [_vp, _vp, _vp, ctypes.POINTER(_i), _vp]),
    "rx_attend_suffix": (_i, [_vp, _i, _vp, _vp, _vp, _i, _vp, _vp]),
    "rx_attend_batch": (_i, [_vp, _i, _vp, _vp, _vp, _i, _vp, ctypes.POINTER(RxStreamBatch), _vp]),
    "rx_ada_gamma": (_i, [_vp, _vp, _i, _i, _i, _vp, _vp, _i, _vp, _vp, _i, _i, _vp, _vp]),
    "rx_adarmsnorm": (_i, [_vp, _vp, _i, _i, _f, _vp, _vp]),
    "rx_get_state": (_i, [_vp, ctypes.POINTER(_i), ctypes.POINTER(_i),
                          ctypes.POINTER(ctypes.c_longlong), _vp]),
    "rx_debug_window": (_i, [_vp, ctypes.POINTER(_i), ctypes.POINTER(_i), _vp]),
    "rx_export_window": (_i, [_vp, _i, _vp, _vp, _vp]),
    "rx_check_device_error": (_i, [_vp, ctypes.POINTER(_i), _vp]),
    "rx_set_attn_splits": (_i, [_vp, _i]),
    "rx_set_attn_dparts": (_i, [_vp, _i]),
    "rx_debug_inject_timeout": (_i, [_vp, _i]),
    "rx_debug_choose_partition": (_i, [_i, _i, _i, _i, _i, _i, _i, ctypes.POINTER(_i),
                                       ctypes.POINTER(_i), ctypes.POINTER(_i), ctypes.POINTER(_i)]),
    "rx_launch_count": (ctypes.c_longlong, []),
    "rx_status_str": (ctypes.c_char_p, [_i]),
    "rx_last_error": (ctypes.c_char_p, []),
    "rx_attend_regions_static": (_i, [_vp, _i, _i, _i, _i, _vp, _vp, _i, _vp, _vp, _i,
                                      _vp, _vp, _i, _vp, _vp]),
    "rx_attend_suffix_block_causal": (_i, [_vp, _i, _vp, _vp, _vp, _i, _i, _vp, _vp]),
    "rx_tail_append": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _vp, _vp]),
    "rx_snapshot_bytes": (_i, [_vp, ctypes.POINTER(ctypes.c_longlong)]),
    "rx_snapshot": (_i, [_vp, _vp, _vp]),
    "rx_restore": (_i, [_vp, _vp, _vp]),
    "rx_push_frame_async": (_i, [_vp, _vp, _vp, ctypes.POINTER(_i), _vp, _vp]),
    "rx_attend_suffix_norms": (_i, [_vp, _i, _vp, _vp, _vp, _i, _vp, ctypes.POINTER(RxNormRows), _i, _vp]),
    "rx_attend_batch_norms": (_i, [_vp, _i, _vp, _vp, _vp, _i, _vp, ctypes.POINTER(RxStreamBatch),
                                   ctypes.POINTER(RxNormRows), _i, _vp]),
    "rx_tail_append_quant": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _vp]),
    "rx_attend_streams_quant": (_i, [_vp, _i, ctypes.POINTER(RxQuantStreams), _vp]),
    "rx_debug_choose_stream_partition": (_i, [_i, _i, ctypes.c_longlong, _i, _i, ctypes.POINTER(_i),
                                              ctypes.POINTER(_i)]),
    "rx_rotate_heads": (_i, [_vp, ctypes.c_longlong, _i, ctypes.POINTER(RxHeads), _vp, _vp, _vp, _vp, _vp]),
    "rx_rotate_heads_paged": (_i, [_vp, ctypes.c_longlong, _i, ctypes.POINTER(RxHeads), _vp, _vp,
                                   ctypes.POINTER(RxPages), _vp, _vp, _vp, _vp, _vp]),
    "rx_attend_pages": (_i, [_vp, _i, _vp, _i, _i, _i, _i, ctypes.POINTER(RxPages), _vp, _vp, _vp, _vp, _vp, _vp,
                             ctypes.c_longlong, _vp]),
    "rx_attend_pages_workspace": (_i, [_i, _i, _i, _i, ctypes.POINTER(ctypes.c_longlong)]),
    "rx_weigh_pages": (_i, [_vp, _vp, _i, _i, _i, _i, ctypes.POINTER(RxPages), _vp, _vp, _vp, _f, _vp, _vp, ctypes.c_longlong, _vp]),
    "rx_weigh_pages_workspace": (_i, [_i, _i, _i, ctypes.POINTER(ctypes.c_longlong)]),
    "rx_evict_pages": (_i, [ctypes.POINTER(RxPages), _i, _i, _vp, _i, _i, _i, _vp, _i, _vp, _vp, _vp, _vp]),
    "rx_debug_page_plan": (_i, [_i] * 7 + [ctypes.POINTER(ctypes.c_longlong), ctypes.POINTER(_i)]),
    "rx_verify_drafts": (_i, [_vp, _vp, _i, _vp, _vp, _vp, _vp, _i, _i, _i, _vp, _vp, _vp, _vp, _vp]),
}
for _name, (_res, _args) in _sigs.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args


class RxError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _lib.rx_last_error().decode(errors="replace")
        super().__init__("%s failed: %s: %s" % (where, STATUS_NAMES.get(status, status), msg))


def _check(status: int, where: str) -> None:
    if status != RX_OK:
        raise RxError(status, where)


def _stream(stream=None) -> int:
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _ptr(t: Optional[torch.Tensor], dtype=torch.bfloat16, name: str = "tensor",
         device: bool = True) -> Optional[int]:
    if t is None:
        return None
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if device and not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    return t.data_ptr()


def _shape(t: Optional[torch.Tensor], shape, name: str) -> None:
    """Refuse a tensor whose shape differs from the one the library will
    assume from the sizes it is given (it would read or write past the
    caller's buffer)."""
    if t is not None and tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))


def _addresses(dev: int, *specs) -> list:
    """The addresses of tensors (or None) that the library will take to be
    contiguous, of these types and shapes, on the current device `dev`:
    (tensor, dtype, shape, name) each.  Anything else is refused, shapes
    first.  (One test for the good case: a call of the language streams' entry
    points is short beside a check for each property.)"""
    out = []
    for t, dtype, shape, _ in specs:
        if t is None:
            out.append(None)
        elif t.shape == shape and t.dtype is dtype and t.is_contiguous() and t.get_device() == dev:
            out.append(t.data_ptr())
        else:
            break
    else:
        return out
    for t, _, shape, name in specs:
        _shape(t, shape, name)
    for t, dtype, _, name in specs:
        _ptr(t, dtype, name)
    for t, _, _, name in specs:
        if t is not None and t.get_device() != dev:
            raise ValueError("%s must be on the current device (cuda:%d), got %s" % (name, dev, t.device))
    raise ValueError("tensors changed while they were checked")


def _here(stream) -> Tuple[int, int]:
    """The current device, or -2 without one, and the address of `stream` (or
    of that device's current stream)."""
    try:
        dev = torch.cuda.current_device()
    except (RuntimeError, AssertionError):   # no device: every tensor is refused
        dev = -2
    if stream is not None:
        return dev, stream.cuda_stream
    return dev, torch._C._cuda_getCurrentRawStream(dev) if dev >= 0 else 0


def _outputs(stream):
    """Where a call's own outputs are allocated: on the stream that writes
    them, so that their memory is not in use by work still pending elsewhere."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _norm_jobs(norms) -> Tuple[Optional[ctypes.Array], int]:
    """norms: a sequence of (x [rows][d] bf16, gamma [d] fp32, eps, y [rows][d]
    bf16) -> the C array of rx_norm_rows (or None) and its length."""
    if not norms:
        return None, 0
    if len(norms) > MAX_NORM_JOBS:
        raise ValueError("at most %d norm jobs per launch" % MAX_NORM_JOBS)
    arr = (RxNormRows * len(norms))()
    for i, (x, gamma, eps, y) in enumerate(norms):
        rows, d = x.shape
        _shape(gamma, (d,), "gamma")
        _shape(y, x.shape, "y")
        arr[i] = RxNormRows(_ptr(x, name="x"), _ptr(gamma, torch.float32, "gamma"), _ptr(y, name="y"),
                            rows, d, float(eps))
    return arr, len(norms)


def launch_count() -> int:
    return int(_lib.rx_launch_count())


def choose_partition(t_max: int, units: int, D: int, num_sms: int, max_splits: int,
                     cluster_capacity, splits: int = 0, dparts: int = 0):
    """Test aid: (splits, dparts, fused) of an attention launch, computed on
    the host from the given device figures (rx_debug_choose_partition).
    cluster_capacity: 17 ints, entry c = clusters of c CTAs the device holds."""
    cap = (_i * 17)(*[int(c) for c in cluster_capacity])
    sp, dp, fu = _i(0), _i(0), _i(0)
    _check(_lib.rx_debug_choose_partition(t_max, units, D, num_sms, max_splits, splits, dparts, cap,
                                          ctypes.byref(sp), ctypes.byref(dp), ctypes.byref(fu)),
           "rx_debug_choose_partition")
    return sp.value, dp.value, bool(fu.value)


def choose_stream_partition(t_max: int, units: int, tail_tiles: int, num_sms: int, max_splits: int = 32):
    """Test aid: (splits, tail_sms) of an attention call over language streams
    with 8-bit tails (rx_debug_choose_stream_partition)."""
    sp, ts = _i(0), _i(0)
    _check(_lib.rx_debug_choose_stream_partition(t_max, units, tail_tiles, num_sms, max_splits, ctypes.byref(sp),
                                                 ctypes.byref(ts)), "rx_debug_choose_stream_partition")
    return sp.value, ts.value


def page_plan(n: int, length: int, prefix: int, shared: int, G: int, keys: int, r: int):
    """Test aid: (key tiles before row tile r, that tile's row tile) of a stream in
    attend_pages (rx_debug_page_plan)."""
    before, row_tile = ctypes.c_longlong(0), _i(0)
    _check(_lib.rx_debug_page_plan(n, length, prefix, shared, G, keys, r, ctypes.byref(before), ctypes.byref(row_tile)),
           "rx_debug_page_plan")
    return before.value, row_tile.value


def library_path() -> str:
    return _LIB_PATH


#: Handles of caches that the garbage collector took while the current stream
#: was being captured; freed when the next cache is made outside a capture.
_parked: list = []


def _capturing() -> bool:
    return torch.cuda.is_initialized() and torch.cuda.is_current_stream_capturing()


def _free_parked() -> None:
    while _parked and not _capturing():
        _lib.rx_cache_destroy(_parked.pop())   # (as in __del__, nobody is there to hear of a failure)


class Cache:
    """The partitioned KV store of one stream (rx_cache_t)."""

    def __init__(self, L: int, Hq: int, Hkv: int, D: int, P_cap: int, N: int, F: int,
                 S_cap: int, tail_cap: int = 0, max_req: int = 0, spare_slot: int = 0):
        _free_parked()
        self.cfg = RxConfig(L, Hq, Hkv, D, P_cap, N, F, S_cap, tail_cap, max_req, spare_slot)
        h = _vp()
        _check(_lib.rx_cache_create(ctypes.byref(self.cfg), ctypes.byref(h)), "rx_cache_create")
        self._h = h

    @property
    def handle(self):
        return self._h

    def close(self) -> None:
        """Free the cache's memory (synchronises the device, so not while a
        stream is being captured)."""
        h, self._h = getattr(self, "_h", None), None   # freed whatever the status is
        if h:
            _check(_lib.rx_cache_destroy(h), "rx_cache_destroy")

    def __del__(self):
        try:
            if _capturing():   # collected within a capture, which freeing would end
                h, self._h = getattr(self, "_h", None), None
                if h:
                    _parked.append(h)
            else:
                self.close()
        except Exception:
            pass

    def pin_prefix(self, k: torch.Tensor, v: torch.Tensor, stream=None) -> None:
        c = self.cfg
        P = k.shape[1]
        _shape(k, (c.L, P, c.Hkv, c.D), "k")
        _shape(v, k.shape, "v")
        _check(_lib.rx_pin_prefix(self._h, _ptr(k, name="k", device=False),
                                  _ptr(v, name="v", device=False), P, _stream(stream)),
               "rx_pin_prefix")

    def _frame_shape(self, k: torch.Tensor, v: torch.Tensor) -> None:
        c = self.cfg
        _shape(k, (c.L, c.F, c.Hkv, c.D), "k")
        _shape(v, k.shape, "v")

    def push_frame(self, k: torch.Tensor, v: torch.Tensor, stream=None) -> int:
        self._frame_shape(k, v)
        ev = _i(0)
        _check(_lib.rx_push_frame(self._h, _ptr(k, name="k"), _ptr(v, name="v"),
                                  ctypes.byref(ev), _stream(stream)), "rx_push_frame")
        return ev.value

    def push_frame_async(self, k: torch.Tensor, v: torch.Tensor, producer_stream,
                         consumer_stream) -> int:
        """Push on producer_stream, concurrent with attention on consumer_stream
        (needs spare_slot=1)."""
        self._frame_shape(k, v)
        ev = _i(0)
        _check(_lib.rx_push_frame_async(self._h, _ptr(k, name="k"), _ptr(v, name="v"), ctypes.byref(ev),
                                        producer_stream.cuda_stream, consumer_stream.cuda_stream),
               "rx_push_frame_async")
        return ev.value

    def attend_suffix(self, layer: int, q: torch.Tensor, k_dyn: torch.Tensor, v_dyn: torch.Tensor,
                      out: Optional[torch.Tensor] = None, stream=None,
                      n_state: Optional[int] = None, norms=None) -> torch.Tensor:
        """Eq. 1 for one layer; with n_state, the block-causal variant (the
        first n_state suffix tokens see only their own dynamic keys); with
        norms, a list of up to two (x, gamma, eps, y) AdaRMSNorm jobs run in
        the same launch (rx_attend_suffix_norms)."""
        c = self.cfg
        S = q.shape[0]
        _shape(q, (S, c.Hq, c.D), "q")
        _shape(k_dyn, (S, c.Hkv, c.D), "k_dyn")
        _shape(v_dyn, (S, c.Hkv, c.D), "v_dyn")
        _shape(out, q.shape, "out")
        if out is None:
            out = torch.empty_like(q)
        if norms:
            if n_state is not None:
                raise ValueError("norm jobs run with the plain Eq. 1 call only")
            arr, n = _norm_jobs(norms)
            _check(_lib.rx_attend_suffix_norms(self._h, layer, _ptr(q, name="q"), _ptr(k_dyn, name="k_dyn"),
                                               _ptr(v_dyn, name="v_dyn"), S, _ptr(out, name="out"), arr, n,
                                               _stream(stream)), "rx_attend_suffix_norms")
        elif n_state is None:
            _check(_lib.rx_attend_suffix(self._h, layer, _ptr(q, name="q"), _ptr(k_dyn, name="k_dyn"),
                                         _ptr(v_dyn, name="v_dyn"), S, _ptr(out, name="out"),
                                         _stream(stream)), "rx_attend_suffix")
        else:
            _check(_lib.rx_attend_suffix_block_causal(
                self._h, layer, _ptr(q, name="q"), _ptr(k_dyn, name="k_dyn"), _ptr(v_dyn, name="v_dyn"),
                S, int(n_state), _ptr(out, name="out"), _stream(stream)), "rx_attend_suffix_block_causal")
        return out

    def snapshot_bytes(self) -> int:
        n = ctypes.c_longlong(0)
        _check(_lib.rx_snapshot_bytes(self._h, ctypes.byref(n)), "rx_snapshot_bytes")
        return n.value

    def snapshot(self, dst: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """Copy the cache's state into a uint8 CUDA tensor (allocated if not given)."""
        if dst is None:
            dst = torch.empty(self.snapshot_bytes(), dtype=torch.uint8, device="cuda")
        _check(_lib.rx_snapshot(self._h, _ptr(dst, torch.uint8, "dst"), _stream(stream)), "rx_snapshot")
        return dst

    def restore(self, src: torch.Tensor, stream=None) -> None:
        _check(_lib.rx_restore(self._h, _ptr(src, torch.uint8, "src"), _stream(stream)), "rx_restore")

    def attend_batch(self, layer: int, action=None, lang=None, out_act: Optional[torch.Tensor] = None,
                     out_lang: Optional[torch.Tensor] = None, stream=None, norms=None):
        """One launch for an action suffix and a batch of language streams.

        action: (q [S][Hq][D], k_dyn [S][Hkv][D], v_dyn) or None.
        lang: (q [B][T][Hq][D], k_tail [B][tail_cap][Hkv][D], v_tail,
               tail_len int32 CUDA tensor [B]) or None.
        norms: up to two (x, gamma, eps, y) AdaRMSNorm jobs run in the same
               launch (rx_attend_batch_norms).
        Returns (out_act or None, out_lang or None).
        """
        c = self.cfg
        S, qa, kd, vd = 0, None, None, None
        if action is not None:
            qa, kd, vd = action
            S = qa.shape[0]
            _shape(qa, (S, c.Hq, c.D), "q")
            _shape(kd, (S, c.Hkv, c.D), "k_dyn")
            _shape(vd, (S, c.Hkv, c.D), "v_dyn")
            _shape(out_act, qa.shape, "out_act")
            if out_act is None:
                out_act = torch.empty_like(qa)
        batch = None
        if lang is not None:
            ql, kt, vt, tl = lang
            B = ql.shape[0]
            _shape(ql, (B, ql.shape[1] if ql.dim() > 1 else 0, c.Hq, c.D), "q_lang")
            _shape(kt, (B, c.tail_cap, c.Hkv, c.D), "k_tail")
            _shape(vt, kt.shape, "v_tail")
            _shape(tl, (B,), "tail_len")
            _shape(out_lang, ql.shape, "out_lang")
            if out_lang is None:
                out_lang = torch.empty_like(ql)
            batch = RxStreamBatch(_ptr(ql, name="q_lang"), _ptr(kt, name="k_tail"),
                                  _ptr(vt, name="v_tail"), _ptr(tl, torch.int32, "tail_len"),
                                  _ptr(out_lang, name="out_lang"), ql.shape[0], ql.shape[1])
        if norms:
            arr, n = _norm_jobs(norms)
            _check(_lib.rx_attend_batch_norms(self._h, layer, _ptr(qa, name="q"), _ptr(kd, name="k_dyn"),
                                              _ptr(vd, name="v_dyn"), S, _ptr(out_act, name="out_act"),
                                              ctypes.byref(batch) if batch is not None else None,
                                              arr, n, _stream(stream)), "rx_attend_batch_norms")
        else:
            _check(_lib.rx_attend_batch(self._h, layer, _ptr(qa, name="q"), _ptr(kd, name="k_dyn"),
                                        _ptr(vd, name="v_dyn"), S, _ptr(out_act, name="out_act"),
                                        ctypes.byref(batch) if batch is not None else None,
                                        _stream(stream)), "rx_attend_batch")
        return (out_act if action is not None else None), (out_lang if lang is not None else None)

    def attend_streams_quant(self, layer: int, q: torch.Tensor, k_tail: torch.Tensor, v_tail: torch.Tensor,
                             k_exp: torch.Tensor, v_exp: torch.Tensor, tail_len: torch.Tensor,
                             n_new: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                             stream=None) -> torch.Tensor:
        """Language streams over the shared store and their own 8-bit tails.

        q: bf16 [B][T][Hq][D], the newest n_new[b] <= T tokens of each tail
        (n_new None: T); tails: float8_e4m3fn [B][tail_cap][Hkv][D] with
        uint8 exponents [B][tail_cap][Hkv] (tail_append_quant); tail_len:
        int32 [B], the query tokens' own keys among them.  Query token t sees
        the cached regions and its stream's keys up to its own.  Rows
        t >= n_new[b] of out are left as they were (of a new one: undefined).
        """
        c = self.cfg
        if q.dim() != 4:
            raise ValueError("q must have shape [B][T][Hq][D]")
        B, T = q.shape[:2]
        dev, st = _here(stream)
        if out is None:
            with _outputs(stream):
                out = torch.empty_like(q)
        e4m3, u8, i32, bf16 = torch.float8_e4m3fn, torch.uint8, torch.int32, torch.bfloat16
        rows, tail, exps, each = (B, T, c.Hq, c.D), (B, c.tail_cap, c.Hkv, c.D), (B, c.tail_cap, c.Hkv), (B,)
        ptrs = _addresses(dev, (q, bf16, rows, "q"), (k_tail, e4m3, tail, "k_tail"), (v_tail, e4m3, tail, "v_tail"),
                          (k_exp, u8, exps, "k_exp"), (v_exp, u8, exps, "v_exp"), (tail_len, i32, each, "tail_len"),
                          (n_new, i32, each, "n_new"), (out, bf16, rows, "out"))
        batch = RxQuantStreams(*ptrs, B, T)
        _check(_lib.rx_attend_streams_quant(self._h, layer, ctypes.byref(batch), st), "rx_attend_streams_quant")
        return out

    def attend_pages(self, layer: int, q: torch.Tensor, pages: "Pages", q_start: torch.Tensor, length: torch.Tensor,
                     prefix: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None, lse=None,
                     workspace: Optional[torch.Tensor] = None, stream=None):
        """New tokens of language streams over the shared store of `layer` and
        their own pages (see attend_pages)."""
        return _attend_pages(self, layer, q, pages, q_start, length, prefix, out, lse, workspace, stream)

    def get_state(self, stream=None) -> Tuple[int, int, int]:
        h, v, p = _i(0), _i(0), ctypes.c_longlong(0)
        _check(_lib.rx_get_state(self._h, ctypes.byref(h), ctypes.byref(v), ctypes.byref(p),
                                 _stream(stream)), "rx_get_state")
        return h.value, v.value, p.value

    def debug_window(self, stream=None) -> List[int]:
        slots = (_i * self.cfg.N)()
        valid = _i(0)
        _check(_lib.rx_debug_window(self._h, slots, ctypes.byref(valid), _stream(stream)),
               "rx_debug_window")
        return [slots[i] for i in range(valid.value)]

    def export_window(self, layer: int, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
        valid = len(self.debug_window(stream))
        c = self.cfg
        k = torch.empty((valid * c.F, c.Hkv, c.D), dtype=torch.bfloat16, device="cuda")
        v = torch.empty_like(k)
        if valid:
            _check(_lib.rx_export_window(self._h, layer, _ptr(k), _ptr(v), _stream(stream)),
                   "rx_export_window")
        return k, v

    def check_device_error(self, stream=None) -> int:
        code = _i(0)
        _check(_lib.rx_check_device_error(self._h, ctypes.byref(code), _stream(stream)),
               "rx_check_device_error")
        return code.value

    def set_attn_splits(self, splits: int) -> None:
        _check(_lib.rx_set_attn_splits(self._h, splits), "rx_set_attn_splits")

    def set_attn_dparts(self, dparts: int) -> None:
        _check(_lib.rx_set_attn_dparts(self._h, dparts), "rx_set_attn_dparts")

    def debug_inject_timeout(self, nbytes: int) -> None:
        """Test aid: the next attention launch's first CTA waits for nbytes
        that never arrive, so its bounded waits run out (see rx.h)."""
        _check(_lib.rx_debug_inject_timeout(self._h, nbytes), "rx_debug_inject_timeout")


def ada_gamma(t: torch.Tensor, state: torch.Tensor, W1: torch.Tensor, b1: torch.Tensor,
              W2: torch.Tensor, b2: torch.Tensor, emb_dim: int,
              out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """gamma [n_sets][n_cond][d] for weights W1 [n_sets][hidden][cond], W2 [n_sets][d][hidden]."""
    n_cond = t.shape[0]
    state_dim = state.shape[1] if state.dim() == 2 else 0
    n_sets, hidden, cond = W1.shape
    d = W2.shape[1]
    if cond != emb_dim + state_dim:
        raise ValueError("W1 input width %d != emb_dim + state_dim = %d" % (cond, emb_dim + state_dim))
    _shape(t, (n_cond,), "t")
    _shape(state, (n_cond, state_dim), "state")
    _shape(b1, (n_sets, hidden), "b1")
    _shape(W2, (n_sets, d, hidden), "W2")
    _shape(b2, (n_sets, d), "b2")
    _shape(out, (n_sets, n_cond, d), "gamma")
    if out is None:
        out = torch.empty((n_sets, n_cond, d), dtype=torch.float32, device=t.device)
    _check(_lib.rx_ada_gamma(_ptr(t, torch.float32, "t"), _ptr(state, torch.float32, "state"),
                             n_cond, emb_dim, state_dim, _ptr(W1, name="W1"), _ptr(b1, name="b1"),
                             hidden, _ptr(W2, name="W2"), _ptr(b2, name="b2"), d, n_sets,
                             _ptr(out, torch.float32, "gamma"), _stream(stream)), "rx_ada_gamma")
    return out


def adarmsnorm(x: torch.Tensor, gamma: torch.Tensor, eps: float,
               out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    rows, d = x.shape
    _shape(gamma, (d,), "gamma")
    _shape(out, x.shape, "y")
    if out is None:
        out = torch.empty_like(x)
    _check(_lib.rx_adarmsnorm(_ptr(x, name="x"), _ptr(gamma, torch.float32, "gamma"), rows, d,
                              float(eps), _ptr(out, name="y"), _stream(stream)), "rx_adarmsnorm")
    return out


def attend_regions_static(q: torch.Tensor, k_pin: Optional[torch.Tensor], v_pin: Optional[torch.Tensor],
                          k_win: Optional[torch.Tensor], v_win: Optional[torch.Tensor],
                          k_dyn: Optional[torch.Tensor], v_dyn: Optional[torch.Tensor],
                          out: torch.Tensor, stream=None) -> torch.Tensor:
    """Attention over caller-held regions through rx_attend_regions_static.

    For callers that cannot allocate device memory: the library allocates
    nothing on this path (its scratch is a fixed array inside librx.so), so
    `out` must be supplied.  Regions are [tokens][Hkv][D] bf16 or None.
    """
    S, Hq, D = q.shape
    regions = [(k_pin, v_pin), (k_win, v_win), (k_dyn, v_dyn)]
    for k, v in regions:
        if (k is None) != (v is None):
            raise ValueError("a region needs both its keys and its values (or neither)")
    Hkv = next((k.shape[1] for k, _ in regions if k is not None and k.dim() == 3), 1)
    for (k, v), name in zip(regions, ("pin", "win", "dyn")):
        if k is not None:
            _shape(k, (k.shape[0], Hkv, D), "k_" + name)
            _shape(v, k.shape, "v_" + name)
    _shape(out, q.shape, "out")
    counts = [0 if k is None else k.shape[0] for k, _ in regions]
    ptrs = [(_ptr(k, name="k") if n else None, _ptr(v, name="v") if n else None)
            for (k, v), n in zip(regions, counts)]
    _check(_lib.rx_attend_regions_static(_ptr(q, name="q"), S, Hq, Hkv, D,
                                         ptrs[0][0], ptrs[0][1], counts[0],
                                         ptrs[1][0], ptrs[1][1], counts[1],
                                         ptrs[2][0], ptrs[2][1], counts[2],
                                         _ptr(out, name="out"), _stream(stream)),
           "rx_attend_regions_static")
    return out


def tail_append(k_tail: torch.Tensor, v_tail: torch.Tensor, tail_len: torch.Tensor,
                k_new: torch.Tensor, v_new: torch.Tensor, active: Optional[torch.Tensor] = None,
                overflow: Optional[torch.Tensor] = None, stream=None) -> None:
    """Append one token per (active) stream: tails [B][tail_cap][Hkv][D],
    tail_len int32 [B] (advanced on the device), new tokens [B][Hkv][D]."""
    B, tail_cap, Hkv, D = k_tail.shape
    _shape(v_tail, k_tail.shape, "v_tail")
    _shape(tail_len, (B,), "tail_len")
    _shape(k_new, (B, Hkv, D), "k_new")
    _shape(v_new, (B, Hkv, D), "v_new")
    _shape(active, (B,), "active")
    if overflow is not None and overflow.numel() < 1:
        raise ValueError("overflow must hold one int32")
    _check(_lib.rx_tail_append(_ptr(k_tail, name="k_tail"), _ptr(v_tail, name="v_tail"),
                               _ptr(tail_len, torch.int32, "tail_len"), _ptr(k_new, name="k_new"),
                               _ptr(v_new, name="v_new"), _ptr(active, torch.int32, "active"), B,
                               tail_cap, Hkv, D, _ptr(overflow, torch.int32, "overflow"),
                               _stream(stream)), "rx_tail_append")


def tail_append_quant(k_tail: torch.Tensor, v_tail: torch.Tensor, k_exp: torch.Tensor, v_exp: torch.Tensor,
                      tail_len: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                      n_new: Optional[torch.Tensor] = None, new_len: Optional[torch.Tensor] = None,
                      overflow: Optional[torch.Tensor] = None, stream=None) -> None:
    """Append up to T tokens per stream to 8-bit tails: codes float8_e4m3fn
    [B][tail_cap][Hkv][D], exponents uint8 [B][tail_cap][Hkv] (a code stands
    for code * 2^(exponent - 127)), new tokens bf16 [B][T][Hkv][D], of which
    stream b appends n_new[b] (None: T) at tail_len[b].  tail_len stays as it
    is; new_len, if given, receives the lengths after the append."""
    if k_tail.dim() != 4 or k_new.dim() != 4:
        raise ValueError("tails must have shape [B][tail_cap][Hkv][D] and new tokens [B][T][Hkv][D]")
    tail = B, tail_cap, Hkv, D = tuple(k_tail.shape)
    T = k_new.shape[1]
    exps, new, each = (B, tail_cap, Hkv), (B, T, Hkv, D), (B,)
    e4m3, u8, i32, bf16 = torch.float8_e4m3fn, torch.uint8, torch.int32, torch.bfloat16
    if overflow is not None and overflow.numel() < 1:
        raise ValueError("overflow must hold one int32")
    dev, st = _here(stream)
    kt, vt, ke, ve, tl, nl, kn, vn, nn, ov = _addresses(
        dev, (k_tail, e4m3, tail, "k_tail"), (v_tail, e4m3, tail, "v_tail"), (k_exp, u8, exps, "k_exp"),
        (v_exp, u8, exps, "v_exp"), (tail_len, i32, each, "tail_len"), (new_len, i32, each, "new_len"),
        (k_new, bf16, new, "k_new"), (v_new, bf16, new, "v_new"), (n_new, i32, each, "n_new"),
        (overflow, i32, None if overflow is None else overflow.shape, "overflow"))
    _check(_lib.rx_tail_append_quant(kt, vt, ke, ve, tl, nl, kn, vn, nn, B, T, tail_cap, Hkv, D, ov, st),
           "rx_tail_append_quant")


_PROB_TYPES = {torch.float32: 0, torch.bfloat16: 1}


def verify_drafts(p: torch.Tensor, q: Optional[torch.Tensor], draft: torch.Tensor, u: torch.Tensor, r: torch.Tensor,
                  n_draft: Optional[torch.Tensor] = None, tail_len: Optional[torch.Tensor] = None,
                  new_len: Optional[torch.Tensor] = None, stream=None):
    """Accept or refuse drafted tokens and draw the token that follows them
    (rx_verify_drafts).  p [B][T+1][V] target and q [B][T][V] draft
    probabilities (fp32 or bf16; q None: drafts without probabilities), draft
    int32 [B][T], u fp32 [B][T] and r fp32 [B] uniform in [0, 1), n_draft int32
    [B] (None: T; negative: an idle slot).

    Returns (tokens int32 [B][T+1], n_accept int32 [B], new_len int32 [B]);
    new_len = tail_len + 1 + n_accept, and None without tail_len."""
    if p.dim() != 3 or draft.dim() != 2:
        raise ValueError("p must have shape [B][T+1][V] and draft [B][T]")
    if p.dtype not in _PROB_TYPES:
        raise TypeError("p must be float32 or bfloat16, got %s" % p.dtype)
    B, T = draft.shape
    V = p.shape[2]
    each, i32, f32 = (B,), torch.int32, torch.float32
    if new_len is not None and tail_len is None:
        raise ValueError("new_len needs tail_len")
    dev, st = _here(stream)
    with _outputs(stream):
        tokens = torch.empty((B, T + 1), dtype=i32, device=p.device)
        n_accept = torch.empty(each, dtype=i32, device=p.device)
        if tail_len is not None and new_len is None:
            new_len = torch.empty_like(tail_len)
    pp, qp, dp, up, rp, np_, tl, nl = _addresses(
        dev, (p, p.dtype, (B, T + 1, V), "p"), (q, p.dtype, (B, T, V), "q"), (draft, i32, (B, T), "draft"),
        (u, f32, (B, T), "u"), (r, f32, each, "r"), (n_draft, i32, each, "n_draft"), (tail_len, i32, each, "tail_len"),
        (new_len, i32, each, "new_len"))
    args = (pp, qp, _PROB_TYPES[p.dtype], dp, up, rp, np_, B, T, V, tl, tokens.data_ptr(), n_accept.data_ptr(), nl, st)
    _check(_lib.rx_verify_drafts(*args), "rx_verify_drafts")
    return tokens, n_accept, new_len


class Pages(NamedTuple):
    """One layer's pages of language streams: k, v bf16 [n_pages][page][Hkv][D]
    with pages of 16, 32, 64, 128 or 256 tokens; table int32 [B][max_pages],
    place j of stream b being row j % page of page table[b][j // page]; weight
    fp32 [n_pages][page][Hkv] or None, the attention weight that keys have
    gathered (weigh_pages, evict_pages)."""
    k: torch.Tensor
    v: torch.Tensor
    table: torch.Tensor
    weight: Optional[torch.Tensor] = None


def _pages(dev: int, g: Pages, more=()):
    """The C form of pages and the addresses of further tensors (_addresses)."""
    if g.k.dim() != 4 or g.table.dim() != 2:
        raise ValueError("pages must have shape [n_pages][page][Hkv][D] and their table [B][max_pages]")
    pool, table = g.k.shape, g.table.shape
    bf16, i32 = torch.bfloat16, torch.int32
    ptrs = _addresses(dev, (g.k, bf16, pool, "pages.k"), (g.v, bf16, pool, "pages.v"),
                      (g.weight, torch.float32, pool[:3], "pages.weight"), (g.table, i32, table, "pages.table"), *more)
    return RxPages(*ptrs[:4], pool[0], pool[1], table[1], table[0]), ptrs[4:]


class Heads:
    """What a layer's heads become (rx_heads): Hq query and Hkv key heads of D
    values, normed where their weight (fp32 [D]) is given, then rotated: freq
    fp32 [R/2] holds the pairs' angles per position, the first sections[0] of
    them turn with axis 0 of the positions, the next sections[1] with axis 1 and
    so on.  Pair i is elements (i, i + R/2), or (2i, 2i + 1) with adjacent.  Its
    tensors are checked here, once; calls read what they hold by then."""

    def __init__(self, Hq: int, Hkv: int, D: int, freq: torch.Tensor, sections: Sequence[int] = (),
                 q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 adjacent: bool = False):
        sections = tuple(int(n) for n in sections) or (freq.shape[0],)
        if len(sections) > MAX_AXES:
            raise ValueError("at most %d axes" % MAX_AXES)
        if sum(sections) != freq.shape[0]:
            raise ValueError("the sections %s hold %d pairs, freq %d" % (sections, sum(sections), freq.shape[0]))
        self.Hq, self.Hkv, self.D, self.axes, self.width = Hq, Hkv, D, len(sections), (Hq + 2 * Hkv) * D
        self.freq, self.q_weight, self.k_weight = freq, q_weight, k_weight
        if not freq.is_cuda:
            raise ValueError("freq must be a CUDA tensor")
        dev, f32, each = freq.get_device(), torch.float32, (D,)
        ptrs = _addresses(dev, (freq, f32, freq.shape, "freq"), (q_weight, f32, each, "q_weight"), (k_weight, f32, each, "k_weight"))
        self._device = dev
        self._c = RxHeads(*ptrs, Hq, Hkv, D, len(sections), (_i * MAX_AXES)(*sections), int(bool(adjacent)), float(eps))


def _heads_input(x: torch.Tensor, heads: Heads, pos: torch.Tensor, dev: int):
    """(tokens, row stride) of a projection's rows, which may be apart, and the
    positions as [axes][N]."""
    if x.dim() != 2 or x.shape[1] != heads.width:
        raise ValueError("x must have shape [N][%d], got %s" % (heads.width, tuple(x.shape)))
    if x.dtype is not torch.bfloat16:
        raise TypeError("x must be %s, got %s" % (torch.bfloat16, x.dtype))
    if x.stride(1) != 1:
        raise ValueError("the values of a row of x must be contiguous")
    if x.get_device() != dev or heads._device != dev:
        raise ValueError("x and the heads' tensors must be on the current device (cuda:%d), got %s and cuda:%d"
                         % (dev, x.device, heads._device))
    N = x.shape[0]
    return N, x.stride(0) if N > 1 else heads.width, pos if pos.dim() == 2 else pos.view(1, -1)


def rotate_heads(x: torch.Tensor, heads: Heads, pos: torch.Tensor, q: Optional[torch.Tensor] = None,
                 k: Optional[torch.Tensor] = None, v: Optional[torch.Tensor] = None, stream=None):
    """Norm and rotate the heads of N tokens: x bf16 [N][(Hq + 2*Hkv)*D]
    (queries, keys, values; rows may be apart), pos int32 [axes][N] (or [N]).
    Returns q [N][Hq][D], k and v [N][Hkv][D]."""
    dev, st = _here(stream)
    N, stride, pos = _heads_input(x, heads, pos, dev)
    qs, ks, bf16 = (N, heads.Hq, heads.D), (N, heads.Hkv, heads.D), torch.bfloat16
    pp, qp, kp, vp = _addresses(dev, (pos, torch.int32, (heads.axes, N), "pos"), (q, bf16, qs, "q"), (k, bf16, ks, "k"),
                                (v, bf16, ks, "v"))
    if q is None or k is None or v is None:
        with _outputs(stream):
            q = x.new_empty(qs) if q is None else q
            k = x.new_empty(ks) if k is None else k
            v = x.new_empty(ks) if v is None else v
        qp, kp, vp = q.data_ptr(), k.data_ptr(), v.data_ptr()
    _check(_lib.rx_rotate_heads(x.data_ptr(), stride, N, ctypes.byref(heads._c), pp, qp, kp, vp, st), "rx_rotate_heads")
    return q, k, v


def rotate_heads_paged(x: torch.Tensor, heads: Heads, pos: torch.Tensor, pages: Pages, q_start: torch.Tensor,
                       held: torch.Tensor, q: Optional[torch.Tensor] = None, new_len: Optional[torch.Tensor] = None,
                       overflow: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """rotate_heads with the keys and values stored in pages: the new tokens of
    stream b, [q_start[b], q_start[b+1]) of x, at places from held[b] on, their
    gathered weight set to 0.  held stays as it is; new_len, if given, receives
    the lengths after the step.  Returns q (rows of tokens in no stream are left
    as they were; of a new one: undefined)."""
    dev, st = _here(stream)
    N, stride, pos = _heads_input(x, heads, pos, dev)
    B = pages.table.shape[0]
    qs, i32 = (N, heads.Hq, heads.D), torch.int32
    if overflow is not None and overflow.numel() < 1:
        raise ValueError("overflow must hold one int32")
    if pages.k.shape[2:] != (heads.Hkv, heads.D):
        raise ValueError("pages have heads %s, expected %s" % (tuple(pages.k.shape[2:]), (heads.Hkv, heads.D)))
    g, (pp, qp, sp, hp, np_, op) = _pages(dev, pages, (
        (pos, i32, (heads.axes, N), "pos"), (q, torch.bfloat16, qs, "q"), (q_start, i32, (B + 1,), "q_start"),
        (held, i32, (B,), "held"), (new_len, i32, (B,), "new_len"),
        (overflow, i32, None if overflow is None else overflow.shape, "overflow")))
    if q is None:
        with _outputs(stream):
            q = x.new_empty(qs)
        qp = q.data_ptr()
    _check(_lib.rx_rotate_heads_paged(x.data_ptr(), stride, N, ctypes.byref(heads._c), pp, qp, ctypes.byref(g), sp, hp,
                                      np_, op, st), "rx_rotate_heads_paged")
    return q


def attend_pages_workspace(N: int, Hq: int, Hkv: int, D: int) -> int:
    """Bytes of workspace that attend_pages needs for N new tokens."""
    n = ctypes.c_longlong(0)
    _check(_lib.rx_attend_pages_workspace(N, Hq, Hkv, D, ctypes.byref(n)), "rx_attend_pages_workspace")
    return n.value


#: attend_pages_workspace() by (device, N, Hq, Hkv, D) and weigh_pages_workspace()
#: by (device, N, Hq, Hkv).
_workspace_sizes: dict = {}


def _workspace_size(dev, of, *shape):
    size = _workspace_sizes.get((dev,) + shape)
    if size is None:
        if len(_workspace_sizes) >= 4096:
            _workspace_sizes.clear()
        size = _workspace_sizes[(dev,) + shape] = of(*shape)
    return size


def _attend_pages(cache, layer, q, pages, q_start, length, prefix, out, lse, workspace, stream):
    if q.dim() != 3 or pages.k.dim() != 4:
        raise ValueError("q must have shape [N][Hq][D] and pages [n_pages][page][Hkv][D]")
    if cache is not None and not cache._h:
        raise ValueError("the cache is closed")
    N, Hq, D = q.shape
    B, Hkv = pages.table.shape[0], pages.k.shape[2]
    bf16, f32, i32, u8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
    if pages.k.shape[3] != D or Hkv < 1 or Hq % Hkv:
        raise ValueError("q has heads %s, the pages %s" % ((Hq, D), tuple(pages.k.shape[2:])))
    dev, st = _here(stream)
    wants_lse = lse is not None and lse is not False
    given = lse if wants_lse and lse is not True else None
    rows, each = (N, Hq, D), (B,)
    g, (qp, sp, lp, pp, op, ep, wp) = _pages(dev, pages, (
        (q, bf16, rows, "q"), (q_start, i32, (B + 1,), "q_start"), (length, i32, each, "length"),
        (prefix, i32, each, "prefix"), (out, bf16, rows, "out"), (given, f32, (N, Hq), "lse"),
        (workspace, u8, None if workspace is None else workspace.shape, "workspace")))
    size = 0 if workspace is None else workspace.numel()
    with _outputs(stream):
        if out is None:
            out = torch.empty_like(q)
            op = out.data_ptr()
        if wants_lse and given is None:
            given = torch.empty((N, Hq), dtype=f32, device=q.device)
            ep = given.data_ptr()
        if workspace is None:
            size = _workspace_size(dev, attend_pages_workspace, N, Hq, Hkv, D)
            workspace = torch.empty(size, dtype=u8, device=q.device)
            wp = workspace.data_ptr()
    _check(_lib.rx_attend_pages(None if cache is None else cache._h, layer, qp, N, Hq, Hkv, D, ctypes.byref(g), sp, lp, pp,
                                op, ep, wp, size, st), "rx_attend_pages")
    return (out, given) if wants_lse else out


def attend_pages(q: torch.Tensor, pages: Pages, q_start: torch.Tensor, length: torch.Tensor,
                 prefix: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None, lse=None,
                 workspace: Optional[torch.Tensor] = None, stream=None):
    """Attention of a step's new tokens over their streams' pages (with a shared
    store: Cache.attend_pages).  q bf16 [N][Hq][D], packed: stream b's new tokens
    are rows [q_start[b], q_start[b+1]) (int32 [B+1]) and the newest of its
    length[b] keys (int32 [B]).  A token sees everything before it and itself,
    and the first prefix[b] places (int32 [B] or None).  lse: True, or an fp32
    [N][Hq] tensor, for the logarithm of the sum of the exponentials too: the
    call then returns (out, lse).  Rows of tokens in no stream are left as they
    were (of a new out: undefined).  workspace: uint8, attend_pages_workspace()
    bytes, for this call alone while it runs; allocated if not given."""
    return _attend_pages(None, 0, q, pages, q_start, length, prefix, out, lse, workspace, stream)


def weigh_pages_workspace(N: int, Hq: int, Hkv: int) -> int:
    """Bytes of workspace that weigh_pages needs for N new tokens: 0 for few."""
    n = ctypes.c_longlong(0)
    _check(_lib.rx_weigh_pages_workspace(N, Hq, Hkv, ctypes.byref(n)), "rx_weigh_pages_workspace")
    return n.value


def weigh_pages(q: torch.Tensor, lse: torch.Tensor, pages: Pages, q_start: torch.Tensor, length: torch.Tensor,
                prefix: Optional[torch.Tensor] = None, decay: float = 1.0, out: Optional[torch.Tensor] = None,
                workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Add the attention weight of a step's new tokens to the keys that they saw:
    out = decay * pages.weight + the sum of exp(score - lse), for every key of a
    stream with new tokens (rx_weigh_pages).  Arguments as of attend_pages, lse
    its second result.  out: fp32 like pages.weight (None: in place).  workspace:
    uint8, weigh_pages_workspace() bytes, for this call alone while it runs;
    allocated if not given and needed."""
    if q.dim() != 3 or pages.k.dim() != 4:
        raise ValueError("q must have shape [N][Hq][D] and pages [n_pages][page][Hkv][D]")
    N, Hq, D = q.shape
    B, Hkv = pages.table.shape[0], pages.k.shape[2]
    f32, i32, each = torch.float32, torch.int32, (B,)
    if pages.k.shape[3] != D or Hkv < 1 or Hq % Hkv:
        raise ValueError("q has heads %s, the pages %s" % ((Hq, D), tuple(pages.k.shape[2:])))
    if out is None:
        out = pages.weight
    if out is None:
        raise ValueError("the pages have no weight")
    dev, st = _here(stream)
    g, (qp, ep, sp, lp, pp, op, wp) = _pages(dev, pages, (
        (q, torch.bfloat16, (N, Hq, D), "q"), (lse, f32, (N, Hq), "lse"), (q_start, i32, (B + 1,), "q_start"),
        (length, i32, each, "length"), (prefix, i32, each, "prefix"), (out, f32, pages.k.shape[:3], "out"),
        (workspace, torch.uint8, None if workspace is None else workspace.shape, "workspace")))
    size = _workspace_size(dev, weigh_pages_workspace, N, Hq, Hkv) if workspace is None else workspace.numel()
    if workspace is None and size:
        with _outputs(stream):
            workspace = torch.empty(size, dtype=torch.uint8, device=q.device)
        wp = workspace.data_ptr()
    _check(_lib.rx_weigh_pages(qp, ep, N, Hq, Hkv, D, ctypes.byref(g), sp, lp, pp, float(decay), op, wp, size, st),
           "rx_weigh_pages")
    return out


def evict_pages(pages: Pages, length: torch.Tensor, budget: int, sink: int = 0, recent: int = 0,
                to: Optional[torch.Tensor] = None, new_len: Optional[torch.Tensor] = None,
                kept: Optional[torch.Tensor] = None, overflow: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Cut streams of more than `budget` keys back to it: every K/V head keeps its
    first `sink` keys, its last `recent` and the heaviest between them by
    pages.weight, closed up in their order, in place or in the pages of the table
    `to` int32 [B][...] (rx_evict_pages).  length int32 [B]; new_len, if given,
    receives the lengths afterwards and may be length itself.  Returns kept int32
    [B][Hkv][budget]: the old place of every new one, -1 behind the last."""
    if pages.k.dim() != 4 or pages.table.dim() != 2:
        raise ValueError("pages must have shape [n_pages][page][Hkv][D] and their table [B][max_pages]")
    if pages.weight is None:
        raise ValueError("the pages have no weight")
    if to is not None and (to.dim() != 2 or to.shape[0] != pages.table.shape[0]):
        raise ValueError("to must have shape [B][pages], got %s" % (tuple(to.shape),))
    if overflow is not None and overflow.numel() < 1:
        raise ValueError("overflow must hold one int32")
    B, (Hkv, D), i32 = pages.table.shape[0], pages.k.shape[2:], torch.int32
    dev, st = _here(stream)
    g, (lp, tp, np_, kp, op) = _pages(dev, pages, (
        (length, i32, (B,), "length"), (to, i32, None if to is None else to.shape, "to"), (new_len, i32, (B,), "new_len"),
        (kept, i32, (B, Hkv, budget), "kept"), (overflow, i32, None if overflow is None else overflow.shape, "overflow")))
    if kept is None:
        with _outputs(stream):
            kept = torch.empty((B, Hkv, max(0, budget)), dtype=i32, device=pages.k.device)
        kp = kept.data_ptr()
    _check(_lib.rx_evict_pages(ctypes.byref(g), Hkv, D, lp, sink, recent, budget, tp, 0 if to is None else to.shape[1], np_,
                               kp, op, st), "rx_evict_pages")
    return kept
