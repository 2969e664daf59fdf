"""ctypes binding of libnsa_b200.so.

Argument marshalling only: each function passes device pointers (torch tensors
or raw integers), sizes and the stream to the C entry point of the same name
and raises ``NsaError`` on a non-zero status.  Every step of the computation
runs in the library's CUDA kernels; importing this module fails loudly when
the library has not been built.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

from .workloads import Workload

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libnsa_b200.so")
if not os.path.exists(_LIB_PATH):
    raise ImportError(f"{_LIB_PATH} is missing: build it with "
                      "`python -m dynamic_block_sparse_scoring_b200.build` (needs nvcc)")
lib = ctypes.CDLL(_LIB_PATH)

NSA_BR_CMP, NSA_BR_SEL, NSA_BR_WIN, NSA_PER_HEAD_SELECT = 1, 2, 4, 8
NSA_SCORE_PROB, NSA_SCORE_CMP, NSA_SINK_SHIFT, NSA_DEBUG_CHECKS = 16, 32, 16, 64
STATUS = {0: "NSA_OK", 1: "NSA_ERR_INVALID_ARG", 2: "NSA_ERR_UNSUPPORTED", 3: "NSA_ERR_WORKSPACE",
          4: "NSA_ERR_CUDA", 5: "NSA_ERR_TIMEOUT"}


class NsaConfig(ctypes.Structure):
    """Mirror of ``nsa_config`` in include/nsa.h."""
    _fields_ = [("batch", ctypes.c_int32), ("seqlen_q", ctypes.c_int32),
                ("seqlen_kv", ctypes.c_int32), ("q_pos0", ctypes.c_int32),
                ("h_q", ctypes.c_int32), ("h_kv", ctypes.c_int32), ("d_qk", ctypes.c_int32),
                ("d_v", ctypes.c_int32), ("sel_block", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("window", ctypes.c_int32), ("cmp_block", ctypes.c_int32),
                ("cmp_stride", ctypes.c_int32), ("scale", ctypes.c_float),
                ("flags", ctypes.c_uint32)]


class NsaWindowConfig(ctypes.Structure):
    """Mirror of ``nsa_window_config`` in include/nsa.h."""
    _fields_ = [("batch", ctypes.c_int32), ("seqlen_q", ctypes.c_int32),
                ("seqlen_kv", ctypes.c_int32), ("q_pos0", ctypes.c_int32),
                ("h_q", ctypes.c_int32), ("h_kv", ctypes.c_int32), ("d_qk", ctypes.c_int32),
                ("d_v", ctypes.c_int32), ("window", ctypes.c_int32), ("sink", ctypes.c_int32),
                ("scale", ctypes.c_float), ("flags", ctypes.c_uint32)]


class NsaPagedConfig(ctypes.Structure):
    """Mirror of ``nsa_paged_config`` in include/nsa.h."""
    _fields_ = [("batch", ctypes.c_int32), ("seqlen_q", ctypes.c_int32), ("h_q", ctypes.c_int32),
                ("h_kv", ctypes.c_int32), ("d_qk", ctypes.c_int32), ("d_v", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("n_pages", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("window", ctypes.c_int32), ("sink", ctypes.c_int32),
                ("scale", ctypes.c_float), ("flags", ctypes.c_uint32)]


class NsaError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        msg = lib.nsa_status_string(status).decode()
        if status == 4:
            msg += ": " + lib.nsa_last_cuda_error().decode()
        super().__init__(f"{fn} returned {status} ({msg})")


_vp, _sz = ctypes.c_void_p, ctypes.c_size_t
_cfgp = ctypes.POINTER(NsaConfig)
_wcfgp = ctypes.POINTER(NsaWindowConfig)
_pcfgp = ctypes.POINTER(NsaPagedConfig)
_SIGS = {
    "nsa_workspace_size": [_cfgp, ctypes.POINTER(_sz)],
    "nsa_workspace_size_min": [_cfgp, ctypes.POINTER(_sz)],
    "nsa_pool_kv": [_cfgp, _vp, _vp, _vp, _vp, _vp, _vp],
    "nsa_append_kv": [_cfgp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp],
    "nsa_score_blocks": [_cfgp, _vp, _vp, _vp, _vp],
    "nsa_topk_select": [_cfgp, _vp, _vp, _vp, _vp, _vp],
    "nsa_score_blocks_ex": [_cfgp, _vp, _vp, _vp, _vp, _vp],
    "nsa_topk_select_ex": [_cfgp, _vp, _vp, _vp, _vp, _vp, _vp],
    "nsa_sparse_attn_fwd": [_cfgp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp],
    "nsa_sparse_attn_fwd_noalloc": [_cfgp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp],
    "nsa_get_device_status": [ctypes.POINTER(ctypes.c_int32)],
    "nsa_attn_plan": [_cfgp, ctypes.c_int, _sz, ctypes.POINTER(ctypes.c_int32),
                      ctypes.POINTER(ctypes.c_int32)],
    "nsa_timing_enable": [ctypes.c_int32],
    "nsa_check_bounded_wait": [ctypes.c_uint64, _vp],
    "nsa_set_wait_limit_ns": [ctypes.c_uint64],
    "nsa_bwd_workspace_size": [_cfgp, ctypes.POINTER(_sz)],
    "nsa_sparse_attn_bwd": [_cfgp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                            _sz, _vp],
    "nsa_timing_read": [ctypes.c_int32, ctypes.POINTER(ctypes.c_float),
                        ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(ctypes.c_int32)],
    "nsa_window_attn_fwd": [_wcfgp, _vp, _vp, _vp, _vp, _vp, _vp],
    "nsa_window_bwd_workspace_size": [_wcfgp, ctypes.POINTER(_sz)],
    "nsa_window_attn_bwd": [_wcfgp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp],
    "nsa_paged_workspace_size": [_pcfgp, ctypes.POINTER(_sz)],
    "nsa_paged_attn_fwd": [_pcfgp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp],
    "nsa_paged_append_workspace_size": [_pcfgp, ctypes.POINTER(_sz)],
    "nsa_paged_append": [_pcfgp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp],
    "nsa_pages_fork": [_pcfgp, ctypes.c_int32, _vp, _vp, _vp, _vp, _vp, _vp, _vp],
    "nsa_pages_free": [_pcfgp, ctypes.c_int32, _vp, _vp, _vp, _vp, _vp, _vp, _vp],
    "nsa_pages_compact_workspace_size": [_pcfgp, ctypes.POINTER(_sz)],
    "nsa_pages_compact": [_pcfgp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp],
}
for _name, _args in _SIGS.items():
    _f = getattr(lib, _name)
    _f.argtypes = _args
    _f.restype = ctypes.c_int
lib.nsa_status_string.argtypes = [ctypes.c_int]
lib.nsa_status_string.restype = ctypes.c_char_p
lib.nsa_last_cuda_error.argtypes = []
lib.nsa_last_cuda_error.restype = ctypes.c_char_p

EXPORTS = list(_SIGS) + ["nsa_status_string", "nsa_last_cuda_error"]


def config(wl: Workload, **override) -> NsaConfig:
    """nsa_config for a workload (fields may be overridden by keyword)."""
    f = dict(batch=wl.batch, seqlen_q=wl.seqlen_q, seqlen_kv=wl.seqlen_kv, q_pos0=wl.q_pos0,
             h_q=wl.h_q, h_kv=wl.h_kv, d_qk=wl.d_qk, d_v=wl.d_v, sel_block=wl.sel_block,
             top_k=wl.top_k, window=wl.window, cmp_block=wl.cmp_block,
             cmp_stride=wl.cmp_stride, scale=wl.scale, flags=wl.flags)
    f.update(override)
    return NsaConfig(**f)


def _ptr(x) -> Optional[int]:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream if torch.cuda.is_available() else None
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn: str, status: int):
    if status != 0:
        raise NsaError(fn, status)


def nsa_status_string(status: int) -> str:
    return lib.nsa_status_string(status).decode()


PATHS = {0: "rowwise", 1: "query-major", 2: "block-major", 3: "split-k", 4: "decode"}


def nsa_attn_plan(cfg: NsaConfig, select_inside: bool, ws_bytes: int):
    """(path name, kernels launched) nsa_sparse_attn_fwd uses for this call shape."""
    path, n = ctypes.c_int32(0), ctypes.c_int32(0)
    _check("nsa_attn_plan", lib.nsa_attn_plan(ctypes.byref(cfg), int(select_inside), ws_bytes,
                                              ctypes.byref(path), ctypes.byref(n)))
    return PATHS[path.value], n.value


def nsa_bwd_workspace_size(cfg: NsaConfig) -> int:
    n = _sz(0)
    _check("nsa_bwd_workspace_size", lib.nsa_bwd_workspace_size(ctypes.byref(cfg), ctypes.byref(n)))
    return n.value


def nsa_sparse_attn_bwd(cfg, q, k, v, kcmp, vcmp, gates, idx, d_out, dq, dk, dv, dgates=None,
                        workspace=None, ws_bytes=0, stream=None):
    _check("nsa_sparse_attn_bwd",
           lib.nsa_sparse_attn_bwd(ctypes.byref(cfg), _ptr(q), _ptr(k), _ptr(v), _ptr(kcmp),
                                   _ptr(vcmp), _ptr(gates), _ptr(idx), _ptr(d_out), _ptr(dq),
                                   _ptr(dk), _ptr(dv), _ptr(dgates), _ptr(workspace), ws_bytes,
                                   _stream(stream)))


def nsa_check_bounded_wait(limit_ns: int, stream=None):
    _check("nsa_check_bounded_wait", lib.nsa_check_bounded_wait(limit_ns, _stream(stream)))


def nsa_set_wait_limit_ns(limit_ns: int):
    _check("nsa_set_wait_limit_ns", lib.nsa_set_wait_limit_ns(limit_ns))


def nsa_get_device_status() -> int:
    """Reads and clears the device status word (0 = OK, 5 = a bounded wait timed out)."""
    v = ctypes.c_int32(0)
    _check("nsa_get_device_status", lib.nsa_get_device_status(ctypes.byref(v)))
    return v.value


TIMING_MAX_STAGES = 8


def nsa_timing_enable(on: bool):
    """Start / stop recording stage events in this thread's nsa_sparse_attn_fwd calls."""
    _check("nsa_timing_enable", lib.nsa_timing_enable(int(bool(on))))


def nsa_timing_read():
    """[(stage name, ms)] of this thread's most recent timed nsa_sparse_attn_fwd call."""
    ms = (ctypes.c_float * TIMING_MAX_STAGES)()
    names = (ctypes.c_char_p * TIMING_MAX_STAGES)()
    n = ctypes.c_int32(0)
    _check("nsa_timing_read", lib.nsa_timing_read(TIMING_MAX_STAGES, ms, names, ctypes.byref(n)))
    return [(names[i].decode(), float(ms[i])) for i in range(min(n.value, TIMING_MAX_STAGES))]


def nsa_workspace_size(cfg: NsaConfig) -> int:
    n = _sz(0)
    _check("nsa_workspace_size", lib.nsa_workspace_size(ctypes.byref(cfg), ctypes.byref(n)))
    return n.value


def nsa_workspace_size_min(cfg: NsaConfig) -> int:
    n = _sz(0)
    _check("nsa_workspace_size_min", lib.nsa_workspace_size_min(ctypes.byref(cfg), ctypes.byref(n)))
    return n.value


def nsa_pool_kv(cfg, k, v, kbar, kcmp=None, vcmp=None, stream=None):
    _check("nsa_pool_kv", lib.nsa_pool_kv(ctypes.byref(cfg), _ptr(k), _ptr(v), _ptr(kbar),
                                          _ptr(kcmp), _ptr(vcmp), _stream(stream)))


def nsa_append_kv(cfg, k, v, k_new, v_new, kbar=None, kcmp=None, vcmp=None, stream=None):
    """Append cfg.seqlen_q tokens per sequence at KV position cfg.q_pos0 and refresh the
    pooled tokens they complete (cfg.seqlen_kv = cache rows per plane)."""
    _check("nsa_append_kv", lib.nsa_append_kv(ctypes.byref(cfg), _ptr(k), _ptr(v), _ptr(k_new),
                                              _ptr(v_new), _ptr(kbar), _ptr(kcmp), _ptr(vcmp),
                                              _stream(stream)))


def nsa_score_blocks_ex(cfg, q, kbar, kcmp, scores, stream=None):
    _check("nsa_score_blocks_ex", lib.nsa_score_blocks_ex(ctypes.byref(cfg), _ptr(q), _ptr(kbar),
                                                          _ptr(kcmp), _ptr(scores), _stream(stream)))


def nsa_topk_select_ex(cfg, q, kbar, kcmp, scores, idx, stream=None):
    _check("nsa_topk_select_ex", lib.nsa_topk_select_ex(ctypes.byref(cfg), _ptr(q), _ptr(kbar),
                                                        _ptr(kcmp), _ptr(scores), _ptr(idx),
                                                        _stream(stream)))


def nsa_score_blocks(cfg, q, kbar, scores, stream=None):
    _check("nsa_score_blocks", lib.nsa_score_blocks(ctypes.byref(cfg), _ptr(q), _ptr(kbar),
                                                    _ptr(scores), _stream(stream)))


def nsa_topk_select(cfg, q, kbar, scores, idx, stream=None):
    _check("nsa_topk_select", lib.nsa_topk_select(ctypes.byref(cfg), _ptr(q), _ptr(kbar),
                                                  _ptr(scores), _ptr(idx), _stream(stream)))


def nsa_sparse_attn_fwd(cfg, q, k, v, kbar, kcmp, vcmp, gates, idx, out, workspace=None,
                        ws_bytes=0, stream=None):
    _check("nsa_sparse_attn_fwd",
           lib.nsa_sparse_attn_fwd(ctypes.byref(cfg), _ptr(q), _ptr(k), _ptr(v), _ptr(kbar),
                                   _ptr(kcmp), _ptr(vcmp), _ptr(gates), _ptr(idx), _ptr(out),
                                   _ptr(workspace), ws_bytes, _stream(stream)))


def nsa_sparse_attn_fwd_noalloc(cfg, q, k, v, kbar, kcmp, vcmp, gates, out, stream=None):
    """Forward with internal selection and no workspace (the library's own scratch array)."""
    _check("nsa_sparse_attn_fwd_noalloc",
           lib.nsa_sparse_attn_fwd_noalloc(ctypes.byref(cfg), _ptr(q), _ptr(k), _ptr(v),
                                           _ptr(kbar), _ptr(kcmp), _ptr(vcmp), _ptr(gates),
                                           _ptr(out), _stream(stream)))


# ---------------------------------------------------------------------------
# Buffer shapes and a convenience forward that allocates outputs with torch
# ---------------------------------------------------------------------------

def pooled_shapes(cfg: NsaConfig):
    nb_full = cfg.seqlen_kv // cfg.sel_block
    n_cmp = 0
    if cfg.flags & NSA_BR_CMP and cfg.seqlen_kv >= cfg.cmp_block:
        n_cmp = (cfg.seqlen_kv - cfg.cmp_block) // cfg.cmp_stride + 1
    return {"kbar": (cfg.batch, cfg.h_kv, nb_full, cfg.d_qk),
            "kcmp": (cfg.batch, cfg.h_kv, n_cmp, cfg.d_qk),
            "vcmp": (cfg.batch, cfg.h_kv, n_cmp, cfg.d_v)}


def h_sel(cfg: NsaConfig) -> int:
    return cfg.h_q if cfg.flags & NSA_PER_HEAD_SELECT else cfg.h_kv


def alloc_pooled(cfg: NsaConfig, device):
    sh = pooled_shapes(cfg)
    return {"kbar": torch.empty(sh["kbar"], dtype=torch.float32, device=device),
            "kcmp": torch.empty(sh["kcmp"], dtype=torch.bfloat16, device=device),
            "vcmp": torch.empty(sh["vcmp"], dtype=torch.bfloat16, device=device)}


def forward(cfg: NsaConfig, q, k, v, gates=None, idx=None, stream=None, pooled=None, out=None,
            workspace=None):
    """Pool K/V (unless ``pooled`` is given), select blocks and run the gated forward.

    Returns (out, pooled).  All tensors live on the same CUDA device.
    """
    dev = q.device
    if pooled is None:
        pooled = alloc_pooled(cfg, dev)
        nsa_pool_kv(cfg, k, v, pooled["kbar"], pooled["kcmp"], pooled["vcmp"], stream)
    if out is None:
        out = torch.empty(cfg.batch, cfg.seqlen_q, cfg.h_q, cfg.d_v, dtype=torch.bfloat16,
                          device=dev)
    ws = nsa_workspace_size(cfg)
    if workspace is None:
        workspace = torch.empty(ws, dtype=torch.uint8, device=dev) if ws else None
    else:
        ws = workspace.numel() * workspace.element_size()
    nsa_sparse_attn_fwd(cfg, q, k, v, pooled["kbar"], pooled["kcmp"], pooled["vcmp"], gates, idx,
                        out, workspace, ws, stream)
    return out, pooled


# ---------------------------------------------------------------------------
# Window attention with sink tokens, and the paged cache
# ---------------------------------------------------------------------------

def _counts(counts: int):
    """counts: the bitwise or of a configuration's counts.  ctypes would take a count of 2^31 or more
    modulo 2^32 (negative ones are refused by the entry points)."""
    if counts >> 31 > 0:
        raise ValueError("a count of the configuration does not fit 31 bits")


_I32_MAX = 2 ** 31 - 1          # a window or a number of sinks beyond it covers every key, as this does


def window_config(batch, seqlen_q, seqlen_kv, h_q, h_kv, d_qk, d_v, window, sink=0, q_pos0=0,
                  scale=None) -> NsaWindowConfig:
    """nsa_window_config (scale: 1/sqrt(d_qk) unless given)."""
    _counts(batch | seqlen_q | seqlen_kv | q_pos0 | h_q | h_kv | d_qk | d_v)
    return NsaWindowConfig(batch, seqlen_q, seqlen_kv, q_pos0, h_q, h_kv, d_qk, d_v,
                           min(window, _I32_MAX), min(sink, _I32_MAX),
                           max(d_qk, 1) ** -0.5 if scale is None else scale, 0)


def paged_config(batch, seqlen_q, h_q, h_kv, d_qk, d_v, page_size, n_pages, max_pages, window=0,
                 sink=0, scale=None) -> NsaPagedConfig:
    """nsa_paged_config (scale: 1/sqrt(d_qk) unless given)."""
    _counts(batch | seqlen_q | h_q | h_kv | d_qk | d_v | page_size | n_pages | max_pages)
    return NsaPagedConfig(batch, seqlen_q, h_q, h_kv, d_qk, d_v, page_size, n_pages, max_pages,
                          min(window, _I32_MAX), min(sink, _I32_MAX),
                          max(d_qk, 1) ** -0.5 if scale is None else scale, 0)


def nsa_window_attn_fwd(cfg, q, k, v, out, lse=None, stream=None):
    _check("nsa_window_attn_fwd",
           lib.nsa_window_attn_fwd(ctypes.byref(cfg), _ptr(q), _ptr(k), _ptr(v), _ptr(out),
                                   _ptr(lse), _stream(stream)))


def nsa_window_bwd_workspace_size(cfg) -> int:
    n = _sz(0)
    _check("nsa_window_bwd_workspace_size",
           lib.nsa_window_bwd_workspace_size(ctypes.byref(cfg), ctypes.byref(n)))
    return n.value


def nsa_window_attn_bwd(cfg, q, k, v, out, lse, d_out, dq, dk, dv, workspace=None, ws_bytes=0,
                        stream=None):
    _check("nsa_window_attn_bwd",
           lib.nsa_window_attn_bwd(ctypes.byref(cfg), _ptr(q), _ptr(k), _ptr(v), _ptr(out),
                                   _ptr(lse), _ptr(d_out), _ptr(dq), _ptr(dk), _ptr(dv),
                                   _ptr(workspace), ws_bytes, _stream(stream)))


def nsa_paged_workspace_size(cfg) -> int:
    n = _sz(0)
    _check("nsa_paged_workspace_size",
           lib.nsa_paged_workspace_size(ctypes.byref(cfg), ctypes.byref(n)))
    return n.value


def nsa_paged_attn_fwd(cfg, q, k_pages, v_pages, table, lens, out, lse=None, workspace=None,
                       ws_bytes=0, stream=None):
    _check("nsa_paged_attn_fwd",
           lib.nsa_paged_attn_fwd(ctypes.byref(cfg), _ptr(q), _ptr(k_pages), _ptr(v_pages),
                                  _ptr(table), _ptr(lens), _ptr(out), _ptr(lse), _ptr(workspace),
                                  ws_bytes, _stream(stream)))


def nsa_paged_append_workspace_size(cfg) -> int:
    n = _sz(0)
    _check("nsa_paged_append_workspace_size",
           lib.nsa_paged_append_workspace_size(ctypes.byref(cfg), ctypes.byref(n)))
    return n.value


def nsa_paged_append(cfg, k_new, v_new, n_new, k_pages, v_pages, table, lens, ref, short_pages,
                     workspace=None, ws_bytes=0, stream=None):
    _check("nsa_paged_append",
           lib.nsa_paged_append(ctypes.byref(cfg), _ptr(k_new), _ptr(v_new), _ptr(n_new),
                                _ptr(k_pages), _ptr(v_pages), _ptr(table), _ptr(lens), _ptr(ref),
                                _ptr(short_pages), _ptr(workspace), ws_bytes, _stream(stream)))


def nsa_pages_fork(cfg, n, src, dst, table, lens, ref, done, stream=None):
    _check("nsa_pages_fork",
           lib.nsa_pages_fork(ctypes.byref(cfg), n, _ptr(src), _ptr(dst), _ptr(table), _ptr(lens),
                              _ptr(ref), _ptr(done), _stream(stream)))


def nsa_pages_free(cfg, n, rows, keep, table, lens, ref, done, stream=None):
    _check("nsa_pages_free",
           lib.nsa_pages_free(ctypes.byref(cfg), n, _ptr(rows), _ptr(keep), _ptr(table), _ptr(lens),
                              _ptr(ref), _ptr(done), _stream(stream)))


def nsa_pages_compact_workspace_size(cfg) -> int:
    n = _sz(0)
    _check("nsa_pages_compact_workspace_size",
           lib.nsa_pages_compact_workspace_size(ctypes.byref(cfg), ctypes.byref(n)))
    return n.value


def nsa_pages_compact(cfg, k_pages, v_pages, table, lens, ref, remap, n_live, workspace=None,
                      ws_bytes=0, stream=None):
    _check("nsa_pages_compact",
           lib.nsa_pages_compact(ctypes.byref(cfg), _ptr(k_pages), _ptr(v_pages), _ptr(table),
                                 _ptr(lens), _ptr(ref), _ptr(remap), _ptr(n_live),
                                 _ptr(workspace), ws_bytes, _stream(stream)))


def _device(*named):
    """Checks (name, tensor, shape, dtype) tuples: dense tensors of one CUDA device, returned."""
    dev = named[0][1].device
    if dev.type != "cuda":
        raise ValueError(f"{named[0][0]} is on {dev}: all tensors belong on one CUDA device")
    for name, t, shape, dtype in named:
        if t.dtype is dtype and t.shape == shape and t.device == dev and t.is_contiguous():
            continue
        if t.device != dev:
            raise ValueError(f"{name} is on {t.device}: all tensors belong on one CUDA device")
        if t.dtype != dtype or t.shape != shape:
            raise ValueError(f"{name} is {t.dtype} {tuple(t.shape)}: expected {dtype} {tuple(shape)}")
        raise ValueError(f"{name} is not contiguous")
    return dev


def _run(fn, dev, *args):
    """Calls an entry point with the given arguments and dev's current stream; dev becomes the
    current device for the call where it is not."""
    if torch._C._cuda_getDevice() != dev.index:
        with torch.cuda.device(dev):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(dev.index))
    else:
        status = fn(*args, torch._C._cuda_getCurrentRawStream(dev.index))
    if status != 0:
        raise NsaError(fn.__name__, status)


def _size(fn, cfg) -> int:
    n = _sz(0)
    status = fn(cfg, n)
    if status != 0:
        raise NsaError(fn.__name__, status)
    return n.value


_BF16, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def window_forward(cfg: NsaWindowConfig, q, k, v):
    """Window attention with sink tokens on the current stream: (out bf16, lse fp32).  Not recorded by
    autograd, whatever the inputs require: window_backward gives the gradients."""
    B, Tq, Hq, Hkv, Tk, d, dv = (cfg.batch, cfg.seqlen_q, cfg.h_q, cfg.h_kv, cfg.seqlen_kv, cfg.d_qk, cfg.d_v)
    dev = _device(("q", q, (B, Tq, Hq, d), _BF16), ("k", k, (B, Hkv, Tk, d), _BF16),
                  ("v", v, (B, Hkv, Tk, dv), _BF16))
    out = torch.empty_like(q) if dv == d else q.new_empty((B, Tq, Hq, dv))
    lse = q.new_empty((B, Tq, Hq), dtype=_F32)
    _run(lib.nsa_window_attn_fwd, dev, cfg, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
         lse.data_ptr())
    return out, lse


def window_backward(cfg: NsaWindowConfig, q, k, v, out, lse, d_out):
    """Gradients (dq, dk, dv), bf16, of window_forward on the current stream."""
    B, Tq, Hq, Hkv, Tk, d, dv = (cfg.batch, cfg.seqlen_q, cfg.h_q, cfg.h_kv, cfg.seqlen_kv, cfg.d_qk, cfg.d_v)
    o_shape = (B, Tq, Hq, dv)
    dev = _device(("q", q, (B, Tq, Hq, d), _BF16), ("k", k, (B, Hkv, Tk, d), _BF16),
                  ("v", v, (B, Hkv, Tk, dv), _BF16), ("out", out, o_shape, _BF16),
                  ("lse", lse, (B, Tq, Hq), _F32), ("d_out", d_out, o_shape, _BF16))
    n = _size(lib.nsa_window_bwd_workspace_size, cfg)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ws = q.new_empty(n, dtype=_U8)
    _run(lib.nsa_window_attn_bwd, dev, cfg, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
         lse.data_ptr(), d_out.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), ws.data_ptr(), n)
    return dq, dk, dv


def _cache(cfg, k_pages, v_pages):
    plane = (cfg.n_pages, cfg.h_kv, cfg.page_size)
    return (("k_pages", k_pages, plane + (cfg.d_qk,), _BF16),
            ("v_pages", v_pages, plane + (cfg.d_v,), _BF16))


def _books(cfg, table, lens, ref=None):
    t = (("table", table, (cfg.batch, cfg.max_pages), _I32), ("lens", lens, (cfg.batch,), _I32))
    return t if ref is None else t + (("ref", ref, (cfg.n_pages,), _I32),)


def paged_attention(cfg: NsaPagedConfig, q, k_pages, v_pages, table, lens):
    """Attention of the newest cfg.seqlen_q tokens over the paged cache on the current stream:
    (out bf16, lse fp32)."""
    B, Tq, Hq = cfg.batch, cfg.seqlen_q, cfg.h_q
    dev = _device(("q", q, (B, Tq, Hq, cfg.d_qk), _BF16), *_cache(cfg, k_pages, v_pages),
                  *_books(cfg, table, lens))
    n = _size(lib.nsa_paged_workspace_size, cfg)
    out = torch.empty_like(q) if cfg.d_v == cfg.d_qk else q.new_empty((B, Tq, Hq, cfg.d_v))
    lse = q.new_empty((B, Tq, Hq), dtype=_F32)
    ws = q.new_empty(n, dtype=_U8)
    _run(lib.nsa_paged_attn_fwd, dev, cfg, q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
         table.data_ptr(), lens.data_ptr(), out.data_ptr(), lse.data_ptr(), ws.data_ptr(), n)
    return out, lse


def paged_append(cfg: NsaPagedConfig, k_new, v_new, k_pages, v_pages, table, lens, ref, n_new=None):
    """Appends up to cfg.seqlen_q tokens per sequence, in place, on the current stream.  Returns
    short_pages [1] int32 on the device: 0, the pages that were missing, or -1 where a row would outgrow
    the table (then nothing has changed)."""
    new = (cfg.batch, cfg.h_kv, cfg.seqlen_q)
    extra = () if n_new is None else (("n_new", n_new, (cfg.batch,), _I32),)
    dev = _device(("k_new", k_new, new + (cfg.d_qk,), _BF16), ("v_new", v_new, new + (cfg.d_v,), _BF16),
                  *_cache(cfg, k_pages, v_pages), *_books(cfg, table, lens, ref), *extra)
    n = _size(lib.nsa_paged_append_workspace_size, cfg)
    short = lens.new_empty(1)
    ws = lens.new_empty(n, dtype=_U8)
    _run(lib.nsa_paged_append, dev, cfg, k_new.data_ptr(), v_new.data_ptr(),
         None if n_new is None else n_new.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
         table.data_ptr(), lens.data_ptr(), ref.data_ptr(), short.data_ptr(), ws.data_ptr(), n)
    return short


def pages_fork(cfg: NsaPagedConfig, src, dst, table, lens, ref):
    """Rows dst share the pages of rows src; returns done [n] int32 (1: carried out)."""
    n = src.numel()
    dev = _device(("src", src, (n,), _I32), ("dst", dst, (n,), _I32), *_books(cfg, table, lens, ref))
    done = torch.empty_like(src)
    _run(lib.nsa_pages_fork, dev, cfg, n, src.data_ptr(), dst.data_ptr(), table.data_ptr(), lens.data_ptr(),
         ref.data_ptr(), done.data_ptr())
    return done


def pages_free(cfg: NsaPagedConfig, rows, table, lens, ref, keep=None):
    """Rows keep their first keep tokens (None: none); returns done [n] int32."""
    n = rows.numel()
    extra = () if keep is None else (("keep", keep, (n,), _I32),)
    dev = _device(("rows", rows, (n,), _I32), *_books(cfg, table, lens, ref), *extra)
    done = torch.empty_like(rows)
    _run(lib.nsa_pages_free, dev, cfg, n, rows.data_ptr(), None if keep is None else keep.data_ptr(),
         table.data_ptr(), lens.data_ptr(), ref.data_ptr(), done.data_ptr())
    return done


def pages_compact(cfg: NsaPagedConfig, k_pages, v_pages, table, lens, ref):
    """Moves the pages in use to the lowest ids, in place; returns (remap [n_pages], n_live [1])."""
    dev = _device(*_cache(cfg, k_pages, v_pages), *_books(cfg, table, lens, ref))
    n = _size(lib.nsa_pages_compact_workspace_size, cfg)
    remap, n_live = torch.empty_like(ref), lens.new_empty(1)
    ws = lens.new_empty(n, dtype=_U8)
    _run(lib.nsa_pages_compact, dev, cfg, k_pages.data_ptr(), v_pages.data_ptr(), table.data_ptr(),
         lens.data_ptr(), ref.data_ptr(), remap.data_ptr(), n_live.data_ptr(), ws.data_ptr(), n)
    return remap, n_live
