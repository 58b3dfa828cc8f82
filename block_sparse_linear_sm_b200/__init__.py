"""Python binding of the sparse+linear attention C ABI (include/sla.h).

Argument marshalling only: every step of the layer runs in the CUDA kernels of
libsla.so. The functions keep the C names; tensors are torch CUDA tensors (or
raw device addresses as int), the stream is torch's current stream unless one
is given. A missing library raises instead of falling back to anything.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

from . import workloads  # noqa: F401  (seeded inputs; no layer arithmetic)

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsla.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "sla.h")

SLA_OK = 0
SLA_ERR_INVALID_ARG = 1
SLA_ERR_UNSUPPORTED = 2
SLA_ERR_WORKSPACE = 3
SLA_ERR_CUDA = 4
SLA_ERR_DEVICE_TIMEOUT = 5
SLA_ERR_DEVICE_CHECK = 6

SLA_MODE_THREEWAY = 0
SLA_MODE_TOPN_WINDOW = 1

SLA_CACHE_E4M3 = 0
SLA_CACHE_INT8 = 1


class sla_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("B", "H", "H_kv", "N", "N_valid", "d", "block", "mode", "k_h", "k_l", "top_n",
                 "window", "causal", "has_proj", "proj_per_head", "has_gate", "smooth_k",
                 "linear_all", "cos_filter")] + [("scale", ctypes.c_float), ("cos_theta", ctypes.c_float)] + \
        [(n, ctypes.c_int32) for n in ("nsa_branches", "cmp_block", "cmp_stride")]


class sla_cache_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "H", "H_kv", "d", "n_pages", "max_blocks", "kind")] + \
        [("scale", ctypes.c_float)]


class sla_cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("k", "v", "k_scale", "v_scale", "k_mean", "weight", "block_table", "status")]


class SlaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded C-ABI library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m block_sparse_linear_sm_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, S, I32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32
        C = ctypes.POINTER(sla_config)
        L.sla_validate_config.argtypes = [C]
        L.sla_validate_config.restype = ctypes.c_int
        L.sla_workspace_bytes.argtypes = [C]
        L.sla_workspace_bytes.restype = S
        L.sla_route.argtypes = [P, P, C, P, P, P, P, S, P]
        L.sla_route.restype = ctypes.c_int
        L.sla_forward.argtypes = [P, P, P, P, P, C, P, P, P, S, P]
        L.sla_forward.restype = ctypes.c_int
        L.sla_forward_blocks.argtypes = [P, P, P, P, P, C, I32, I32, P, P, P, S, P]
        L.sla_forward_blocks.restype = ctypes.c_int
        L.sla_forward_timed.argtypes = [P, P, P, P, P, C, P, P, P, S, P,
                                        ctypes.POINTER(ctypes.c_void_p), I32]
        L.sla_forward_timed.restype = ctypes.c_int
        L.sla_num_stages.argtypes = [C]
        L.sla_num_stages.restype = I32
        L.sla_stage_name.argtypes = [C, I32]
        L.sla_stage_name.restype = ctypes.c_char_p
        L.sla_check_device_status.argtypes = [P, P, ctypes.POINTER(I32)]
        L.sla_check_device_status.restype = ctypes.c_int
        L.sla_hilbert_order.argtypes = [I32, I32, I32, ctypes.POINTER(I32)]
        L.sla_hilbert_order.restype = ctypes.c_int
        L.sla_permute_tokens.argtypes = [P, P, P, I32, I32, I32, I32, I32, P]
        L.sla_permute_tokens.restype = ctypes.c_int
        L.sla_selftest_wait_timeout.argtypes = [P, S, ctypes.c_int64, P]
        L.sla_selftest_wait_timeout.restype = ctypes.c_int
        L.sla_backward_workspace_bytes.argtypes = [C]
        L.sla_backward_workspace_bytes.restype = S
        bwd = [P, P, P, P, P, C, P, P, P, P, P, P, P, P, S, P, S, P]
        L.sla_backward.argtypes = bwd
        L.sla_backward.restype = ctypes.c_int
        L.sla_backward_timed.argtypes = bwd + [ctypes.POINTER(ctypes.c_void_p), I32]
        L.sla_backward_timed.restype = ctypes.c_int
        L.sla_backward_num_stages.argtypes = [C]
        L.sla_backward_num_stages.restype = I32
        L.sla_backward_stage_name.argtypes = [C, I32]
        L.sla_backward_stage_name.restype = ctypes.c_char_p
        L.sla_status_string.argtypes = [ctypes.c_int]
        L.sla_status_string.restype = ctypes.c_char_p
        L.sla_version.argtypes = []
        L.sla_version.restype = ctypes.c_char_p
        L.sla_forward_host_device_bytes.argtypes = [C, I32]
        L.sla_forward_host_device_bytes.restype = S
        L.sla_forward_host.argtypes = [P, P, P, P, P, C, P, I32, P, S, P, P, P]
        L.sla_forward_host.restype = ctypes.c_int
        L.sla_route_noalloc.argtypes = [P, P, C, P, P, P, P]
        L.sla_route_noalloc.restype = ctypes.c_int
        L.sla_route_noalloc_status.argtypes = [P, ctypes.POINTER(I32)]
        L.sla_route_noalloc_status.restype = ctypes.c_int
        CC, CM = ctypes.POINTER(sla_cache_config), ctypes.POINTER(sla_cache)
        L.sla_cache_validate_config.argtypes = [CC]
        L.sla_cache_validate_config.restype = ctypes.c_int
        L.sla_cache_append.argtypes = [P, P, CC, CM, I32, P, P, P, P]
        L.sla_cache_append.restype = ctypes.c_int
        L.sla_cache_route.argtypes = [P, CC, CM, I32, P, P, I32, P, P]
        L.sla_cache_route.restype = ctypes.c_int
        L.sla_cache_attend_workspace_bytes.argtypes = [CC, I32, I32, I32, I32]
        L.sla_cache_attend_workspace_bytes.restype = S
        L.sla_cache_attend.argtypes = [P, CC, CM, I32, P, P, P, I32, I32, P, P, S, P]
        L.sla_cache_attend.restype = ctypes.c_int
        L.sla_cache_evict_workspace_bytes.argtypes = [CC, I32]
        L.sla_cache_evict_workspace_bytes.restype = S
        L.sla_cache_evict.argtypes = [CC, CM, P, I32, I32, I32, P, P, P, P, P, S, P]
        L.sla_cache_evict.restype = ctypes.c_int
        _lib = L
    return _lib


def make_config(c) -> sla_config:
    """sla_config from any object with the same field names (e.g. workloads.LayerConfig)."""
    cfg = sla_config()
    for name, _ in sla_config._fields_:
        setattr(cfg, name, getattr(c, name))
    return cfg


def _cfg(c) -> sla_config:
    return c if isinstance(c, sla_config) else make_config(c)


def _ptr(x) -> Optional[int]:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if not x.is_cuda:
        raise ValueError("tensor must live on a CUDA device")
    if not x.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return x.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, where: str) -> None:
    if status != SLA_OK:
        raise SlaError(status, where)


def status_string(status: int) -> str:
    return lib().sla_status_string(status).decode()


def sla_status_string(status: int) -> str:
    return status_string(status)


def sla_validate_config(c) -> int:
    return lib().sla_validate_config(ctypes.byref(_cfg(c)))


def sla_workspace_bytes(c) -> int:
    return int(lib().sla_workspace_bytes(ctypes.byref(_cfg(c))))


def sla_num_stages(c) -> int:
    return int(lib().sla_num_stages(ctypes.byref(_cfg(c))))


def sla_stage_names(c) -> list:
    cfg = _cfg(c)
    n = lib().sla_num_stages(ctypes.byref(cfg))
    return [lib().sla_stage_name(ctypes.byref(cfg), i).decode() for i in range(max(n, 0))]


def sla_route(q, k, c, mask_out, crit_idx, neg_idx, ws, stream=None) -> None:
    cfg = _cfg(c)
    ws_bytes = ws.numel() * ws.element_size() if hasattr(ws, "numel") else int(ws[1])
    ws_ptr = _ptr(ws) if hasattr(ws, "numel") else ws[0]
    _check(lib().sla_route(_ptr(q), _ptr(k), ctypes.byref(cfg), _ptr(mask_out), _ptr(crit_idx),
                           _ptr(neg_idx), ws_ptr, ws_bytes, _stream(stream)), "sla_route")


def sla_forward(q, k, v, w_p, w_g, c, out, mask_out, ws, stream=None) -> None:
    cfg = _cfg(c)
    ws_bytes = ws.numel() * ws.element_size()
    _check(lib().sla_forward(_ptr(q), _ptr(k), _ptr(v), _ptr(w_p), _ptr(w_g), ctypes.byref(cfg),
                             _ptr(out), _ptr(mask_out), _ptr(ws), ws_bytes, _stream(stream)),
           "sla_forward")


def sla_forward_blocks(q, k, v, w_p, w_g, c, qb_begin, qb_end, out, mask_out, ws, stream=None) -> None:
    """sla_forward writing only the output rows of query blocks [qb_begin, qb_end)."""
    cfg = _cfg(c)
    ws_bytes = ws.numel() * ws.element_size()
    _check(lib().sla_forward_blocks(_ptr(q), _ptr(k), _ptr(v), _ptr(w_p), _ptr(w_g), ctypes.byref(cfg),
                                    int(qb_begin), int(qb_end), _ptr(out), _ptr(mask_out), _ptr(ws), ws_bytes,
                                    _stream(stream)), "sla_forward_blocks")


def sla_forward_timed(q, k, v, w_p, w_g, c, out, mask_out, ws, events, stream=None) -> None:
    """events: torch.cuda.Event(enable_timing=True) list of length sla_num_stages(c) + 1."""
    cfg = _cfg(c)
    for e in events:
        if e.cuda_event == 0:  # torch creates the CUDA event on first record
            e.record()
    arr = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
    ws_bytes = ws.numel() * ws.element_size()
    _check(lib().sla_forward_timed(_ptr(q), _ptr(k), _ptr(v), _ptr(w_p), _ptr(w_g),
                                   ctypes.byref(cfg), _ptr(out), _ptr(mask_out), _ptr(ws),
                                   ws_bytes, _stream(stream), arr, len(events)),
           "sla_forward_timed")


def _host_ptr(x) -> Optional[int]:
    if isinstance(x, int):
        return x
    if x.is_cuda:
        raise ValueError("tensor must live in host memory")
    if not x.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return x.data_ptr()


def sla_forward_host_device_bytes(c, n_chunks: int) -> int:
    cfg = _cfg(c)
    return int(lib().sla_forward_host_device_bytes(ctypes.byref(cfg), n_chunks))


def sla_forward_host(q_host, k_host, v_host, w_p, w_g, c, out_host, n_chunks, dev, stream=None,
                     h2d_stream=None, d2h_stream=None) -> None:
    """The layer on host tensors (q/k/v/out in host memory, ideally pinned; w_p, w_g and the
    arena ``dev`` of sla_forward_host_device_bytes(c, n_chunks) bytes on the device)."""
    cfg = _cfg(c)
    dev_bytes = dev.numel() * dev.element_size()
    s = _stream(stream)
    _check(lib().sla_forward_host(_host_ptr(q_host), _host_ptr(k_host), _host_ptr(v_host), _ptr(w_p),
                                  _ptr(w_g), ctypes.byref(cfg), _host_ptr(out_host), n_chunks, _ptr(dev),
                                  dev_bytes, s, s if h2d_stream is None else _stream(h2d_stream),
                                  s if d2h_stream is None else _stream(d2h_stream)),
           "sla_forward_host")


def sla_backward_workspace_bytes(c) -> int:
    cfg = _cfg(c)
    return int(lib().sla_backward_workspace_bytes(ctypes.byref(cfg)))


def sla_backward_num_stages(c) -> int:
    cfg = _cfg(c)
    return int(lib().sla_backward_num_stages(ctypes.byref(cfg)))


def sla_backward_stage_names(c) -> list:
    cfg = _cfg(c)
    n = lib().sla_backward_num_stages(ctypes.byref(cfg))
    return [lib().sla_backward_stage_name(ctypes.byref(cfg), i).decode() for i in range(max(n, 0))]


def _bwd_args(q, k, v, w_p, w_g, c, out, dout, dq, dk, dv, dw_p, dw_g, ws, bws, stream):
    return (_ptr(q), _ptr(k), _ptr(v), _ptr(w_p), _ptr(w_g), ctypes.byref(_cfg(c)), _ptr(out), _ptr(dout),
            _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dw_p), _ptr(dw_g), _ptr(ws), ws.numel() * ws.element_size(),
            _ptr(bws), bws.numel() * bws.element_size(), _stream(stream))


def sla_backward(q, k, v, w_p, w_g, c, out, dout, dq, dk, dv, dw_p, dw_g, ws, bws, stream=None) -> None:
    """Gradients of sum(out * dout); ws is the matching sla_forward call's workspace."""
    _check(lib().sla_backward(*_bwd_args(q, k, v, w_p, w_g, c, out, dout, dq, dk, dv, dw_p, dw_g, ws, bws,
                                         stream)), "sla_backward")


def sla_backward_timed(q, k, v, w_p, w_g, c, out, dout, dq, dk, dv, dw_p, dw_g, ws, bws, events,
                       stream=None) -> None:
    """events: torch.cuda.Event(enable_timing=True) list of length sla_backward_num_stages(c) + 1."""
    for e in events:
        if e.cuda_event == 0:
            e.record()
    arr = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
    _check(lib().sla_backward_timed(*_bwd_args(q, k, v, w_p, w_g, c, out, dout, dq, dk, dv, dw_p, dw_g, ws,
                                               bws, stream), arr, len(events)), "sla_backward_timed")


def sla_route_noalloc(q, k, c, mask_out, crit_idx, neg_idx, stream=None) -> None:
    """sla_route without a workspace: its scratch is the library's static device array."""
    cfg = _cfg(c)
    _check(lib().sla_route_noalloc(_ptr(q), _ptr(k), ctypes.byref(cfg), _ptr(mask_out), _ptr(crit_idx),
                                   _ptr(neg_idx), _stream(stream)), "sla_route_noalloc")


def sla_route_noalloc_status(stream=None) -> tuple:
    """(status, detail) of the last sla_route_noalloc on this device, after synchronising the
    stream; clears the status word."""
    detail = ctypes.c_int32(0)
    st = lib().sla_route_noalloc_status(_stream(stream), ctypes.byref(detail))
    return int(st), int(detail.value)


def sla_check_device_status(ws, stream=None) -> tuple:
    """(status, detail) after synchronising the stream; clears the device status word."""
    detail = ctypes.c_int32(0)
    st = lib().sla_check_device_status(_ptr(ws), _stream(stream), ctypes.byref(detail))
    return int(st), int(detail.value)


def sla_selftest_wait_timeout(ws, limit_ns: int, stream=None) -> None:
    """Enqueue the failure-detection self-test: a bounded wait that runs out and is
    recorded in ws's status word (read it with sla_check_device_status)."""
    nbytes = ws.numel() * ws.element_size() if hasattr(ws, "numel") else 256
    _check(lib().sla_selftest_wait_timeout(_ptr(ws), nbytes, int(limit_ns), _stream(stream)),
           "sla_selftest_wait_timeout")


def sla_hilbert_order(t: int, h: int, w: int):
    """Raster indices of the (t, h, w) grid's tokens in Hilbert-curve order (numpy int32)."""
    import numpy as np
    out = np.empty(t * h * w, dtype=np.int32)
    _check(lib().sla_hilbert_order(t, h, w, out.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))),
           "sla_hilbert_order")
    return out


def sla_permute_tokens(x, y, order, inverse: bool = False, stream=None) -> None:
    """y[..., n, :] = x[..., order[n], :] for n < len(order) (inverse: the scatter back);
    x, y: bf16 [..., n_tok, d] CUDA tensors, order: int32 CUDA tensor."""
    n_tok, d = x.shape[-2], x.shape[-1]
    rows = x.numel() // (n_tok * d)
    _check(lib().sla_permute_tokens(_ptr(x), _ptr(y), _ptr(order), order.numel(), rows, n_tok, d,
                                    1 if inverse else 0, _stream(stream)), "sla_permute_tokens")


# ---------------------------------------------------------------------------
# serving the top-n mode: the paged 8-bit cache
# ---------------------------------------------------------------------------

def make_cache_config(c) -> sla_cache_config:
    """sla_cache_config from any object with the same field names (e.g. workloads.CacheConfig)."""
    cfg = sla_cache_config()
    for name, _ in sla_cache_config._fields_:
        setattr(cfg, name, getattr(c, name))
    return cfg


def _cache_cfg(c) -> sla_cache_config:
    return c if isinstance(c, sla_cache_config) else make_cache_config(c)


torch = None  # loaded with the first SlaCache, which every call below needs
_BF16 = _F32 = _I32 = ()


def _load_torch() -> None:
    global torch, _BF16, _F32, _I32
    if torch is None:
        import torch as module
        torch = module
        _BF16, _F32, _I32 = (torch.bfloat16,), (torch.float32,), (torch.int32,)


def _typed(x, name: str, shape, dtypes, index: int):
    """x's address, after checking what the kernels take for granted of it."""
    if x is None:
        return None
    if x.shape != shape or x.dtype not in dtypes or x.get_device() != index or not x.is_contiguous():
        if tuple(x.shape) != tuple(shape):
            raise ValueError(f"{name}: shape {tuple(x.shape)}, expected {tuple(shape)}")
        if x.dtype not in dtypes:
            raise ValueError(f"{name}: dtype {x.dtype}, expected {' or '.join(map(str, dtypes))}")
        if x.get_device() != index:
            raise ValueError(f"{name}: on {x.device}, the cache is on cuda:{index}")
        raise ValueError(f"{name}: must be contiguous")
    return x.data_ptr()


class SlaCache:
    """The buffers of a paged 8-bit cache (sla_cache in include/sla.h). The tensors may be
    changed in place but not replaced (the attributes are read-only): the addresses are taken
    once.

    k, v          1-byte dtype [n_pages, H_kv, 64, d]
    k_scale, v_scale  float32 [n_pages, H_kv]
    k_mean        float32 [n_pages, H_kv, d] or None (sla_cache_route needs it)
    weight        float32 [B, H_kv, 64 * max_blocks] or None (sla_cache_evict needs it;
                  sla_cache_attend adds to it when it is there)
    block_table   int32 [B, max_blocks]
    status        int32 [64], zeroed once (sla_check_device_status(cache.status) reads it)
    """

    __slots__ = ("k", "v", "k_scale", "v_scale", "k_mean", "weight", "block_table", "status", "device", "index",
                 "kind", "shape", "_c")

    def __init__(self, k, v, k_scale, v_scale, k_mean, weight, block_table, status):
        _load_torch()
        if not k.is_cuda:
            raise ValueError("tensor must live on a CUDA device")
        if k.dim() != 4 or block_table.dim() != 2:
            raise ValueError("k: 4 dimensions expected, block_table: 2")
        n_pages, H_kv, block, d = k.shape
        B, max_blocks = block_table.shape
        bytes_, f32, i32 = (torch.uint8, torch.int8, torch.float8_e4m3fn), _F32, _I32
        dev = k.get_device()
        c = sla_cache()
        c.k = _typed(k, "k", (n_pages, H_kv, 64, d), bytes_, dev)
        c.v = _typed(v, "v", (n_pages, H_kv, 64, d), bytes_, dev)
        c.k_scale = _typed(k_scale, "k_scale", (n_pages, H_kv), f32, dev)
        c.v_scale = _typed(v_scale, "v_scale", (n_pages, H_kv), f32, dev)
        c.k_mean = _typed(k_mean, "k_mean", (n_pages, H_kv, d), f32, dev)
        c.weight = _typed(weight, "weight", (B, H_kv, 64 * max_blocks), f32, dev)
        c.block_table = _typed(block_table, "block_table", (B, max_blocks), i32, dev)
        c.status = _typed(status, "status", (64,), i32, dev)
        if v.dtype != k.dtype:
            raise ValueError("k and v must have the same dtype")
        # the element type where the dtype names one (uint8 holds either)
        kind = {torch.int8: SLA_CACHE_INT8, torch.float8_e4m3fn: SLA_CACHE_E4M3}.get(k.dtype)
        for name, x in dict(k=k, v=v, k_scale=k_scale, v_scale=v_scale, k_mean=k_mean, weight=weight,
                            block_table=block_table, status=status, device=k.device, index=dev, kind=kind,
                            shape=(B, H_kv, d, n_pages, max_blocks), _c=c).items():
            object.__setattr__(self, name, x)

    def __setattr__(self, name, value):
        raise AttributeError(f"a cache's {name} cannot be replaced: its address is taken once; "
                             f"write into the tensor, or build another SlaCache")

    def __delattr__(self, name):
        raise AttributeError(f"a cache's {name} cannot be replaced: its address is taken once")

    @classmethod
    def empty(cls, c, device="cuda", weight: bool = True, k_mean: bool = True) -> "SlaCache":
        """A zeroed cache for c whose block table has no page yet (-1 everywhere)."""
        _load_torch()
        dt = torch.float8_e4m3fn if c.kind == SLA_CACHE_E4M3 else torch.int8

        def zeros(*shape, dtype=torch.float32):
            return torch.zeros(*shape, dtype=dtype, device=device)

        return cls(k=zeros(c.n_pages, c.H_kv, 64, c.d, dtype=torch.uint8).view(dt),
                   v=zeros(c.n_pages, c.H_kv, 64, c.d, dtype=torch.uint8).view(dt),
                   k_scale=zeros(c.n_pages, c.H_kv), v_scale=zeros(c.n_pages, c.H_kv),
                   k_mean=zeros(c.n_pages, c.H_kv, c.d) if k_mean else None,
                   weight=zeros(c.B, c.H_kv, 64 * c.max_blocks) if weight else None,
                   block_table=torch.full((c.B, c.max_blocks), -1, dtype=torch.int32, device=device),
                   status=zeros(64, dtype=torch.int32))


def _cache_call(c, cache: SlaCache) -> sla_cache_config:
    """The configuration, after checking that it describes the cache and that the cache's
    device is the current one (the library launches on the current device)."""
    cfg = c if isinstance(c, sla_cache_config) else make_cache_config(c)
    if (cfg.B, cfg.H_kv, cfg.d, cfg.n_pages, cfg.max_blocks) != cache.shape:
        raise ValueError(f"the configuration's (B, H_kv, d, n_pages, max_blocks) "
                         f"{(cfg.B, cfg.H_kv, cfg.d, cfg.n_pages, cfg.max_blocks)} are not the cache's {cache.shape}")
    if cache.kind is not None and cache.kind != cfg.kind:
        raise ValueError("the configuration's kind is not the cache's dtype")
    if cache.index != torch.cuda.current_device():
        raise ValueError(f"the cache is on {cache.device}, the current device is cuda:{torch.cuda.current_device()}")
    return cfg


def _cache_stream(stream, cache: SlaCache) -> int:
    """The given stream's handle, or the current one's without building a Stream object."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(cache.index)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _ws_args(ws, cache: SlaCache):
    if ws.get_device() != cache.index:
        raise ValueError(f"ws: on {ws.device}, the cache is on {cache.device}")
    return _ptr(ws), ws.numel() * ws.element_size()


def sla_cache_validate_config(c) -> int:
    return lib().sla_cache_validate_config(ctypes.byref(_cache_cfg(c)))


def sla_cache_append(k, v, c, cache: SlaCache, lens, n_new=None, lens_out=None, stream=None) -> None:
    """Writes the first n_new[b] rows of k, v (bf16 [B, H_kv, T, d]) behind lens[b] cached tokens."""
    cfg = _cache_call(c, cache)
    dev, bf16, i32 = cache.index, _BF16, _I32
    T = k.shape[2] if k.dim() == 4 else -1
    _check(lib().sla_cache_append(
        _typed(k, "k", (cfg.B, cfg.H_kv, T, cfg.d), bf16, dev), _typed(v, "v", (cfg.B, cfg.H_kv, T, cfg.d), bf16, dev),
        ctypes.byref(cfg), ctypes.byref(cache._c), T, _typed(lens, "lens", (cfg.B,), i32, dev),
        _typed(n_new, "n_new", (cfg.B,), i32, dev), _typed(lens_out, "lens_out", (cfg.B,), i32, dev),
        _cache_stream(stream, cache)), "sla_cache_append")


def sla_cache_route(q, c, cache: SlaCache, lens, n_new, sel, stream=None) -> None:
    """The top_n = sel.shape[2] past blocks of a step's queries q (bf16 [B, H, T, d])."""
    cfg = _cache_call(c, cache)
    dev, i32 = cache.index, _I32
    T = q.shape[2] if q.dim() == 4 else -1
    top_n = sel.shape[2] if sel.dim() == 3 else -1
    _check(lib().sla_cache_route(
        _typed(q, "q", (cfg.B, cfg.H, T, cfg.d), _BF16, dev), ctypes.byref(cfg), ctypes.byref(cache._c),
        T, _typed(lens, "lens", (cfg.B,), i32, dev), _typed(n_new, "n_new", (cfg.B,), i32, dev), top_n,
        _typed(sel, "sel", (cfg.B, cfg.H_kv, top_n), i32, dev), _cache_stream(stream, cache)), "sla_cache_route")


def sla_cache_attend_workspace_bytes(c, T: int, top_n: int = 0, window: int = 0, with_weight: bool = False) -> int:
    return int(lib().sla_cache_attend_workspace_bytes(ctypes.byref(_cache_cfg(c)), T, top_n, window,
                                                      1 if with_weight else 0))


def sla_cache_attend(q, c, cache: SlaCache, lens, n_new, sel, window, out, ws, stream=None) -> None:
    """Attention of a step's queries q (bf16 [B, H, T, d]) over the cache: all of it (sel None,
    window 0), the last `window` tokens (sel None), or the blocks in sel and the window."""
    cfg = _cache_call(c, cache)
    dev, bf16, i32 = cache.index, _BF16, _I32
    T = q.shape[2] if q.dim() == 4 else -1
    top_n = 0 if sel is None else sel.shape[2] if sel.dim() == 3 else -1
    ws_ptr, ws_bytes = _ws_args(ws, cache)
    _check(lib().sla_cache_attend(
        _typed(q, "q", (cfg.B, cfg.H, T, cfg.d), bf16, dev), ctypes.byref(cfg), ctypes.byref(cache._c), T,
        _typed(lens, "lens", (cfg.B,), i32, dev), _typed(n_new, "n_new", (cfg.B,), i32, dev),
        _typed(sel, "sel", (cfg.B, cfg.H_kv, top_n), i32, dev), top_n, int(window),
        _typed(out, "out", (cfg.B, cfg.H, T, cfg.d), bf16, dev), ws_ptr, ws_bytes, _cache_stream(stream, cache)), "sla_cache_attend")


def sla_cache_evict_workspace_bytes(c, budget: int) -> int:
    return int(lib().sla_cache_evict_workspace_bytes(ctypes.byref(_cache_cfg(c)), budget))


def sla_cache_evict(c, cache: SlaCache, lens, budget, n_sink, n_recent, dst_table, weight_out, kept, lens_out, ws,
                    stream=None) -> None:
    """Cuts every sequence to `budget` tokens, those of largest cache.weight; dst_table (int32
    [B, ceil(budget / 64)]) names the pages that receive them (the cache's own or new ones)."""
    cfg = _cache_call(c, cache)
    dev, i32 = cache.index, _I32
    ws_ptr, ws_bytes = _ws_args(ws, cache)
    _check(lib().sla_cache_evict(
        ctypes.byref(cfg), ctypes.byref(cache._c), _typed(lens, "lens", (cfg.B,), i32, dev), int(budget), int(n_sink),
        int(n_recent), _typed(dst_table, "dst_table", (cfg.B, -(-budget // 64)), i32, dev),
        _typed(weight_out, "weight_out", (cfg.B, cfg.H_kv, 64 * cfg.max_blocks), _F32, dev),
        _typed(kept, "kept", (cfg.B, cfg.H_kv, budget), i32, dev), _typed(lens_out, "lens_out", (cfg.B,), i32, dev),
        ws_ptr, ws_bytes, _cache_stream(stream, cache)), "sla_cache_evict")


def sla_version() -> str:
    return lib().sla_version().decode()
