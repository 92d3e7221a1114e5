"""GB300 (sm_103a) attention-prologue kernels -- Python binding of include/kvq.h.

This module only marshals arguments: it checks that tensors are CUDA tensors
(or pinned host tensors, which the kernels then access in place over the
host interconnect) of the expected dtype and layout, takes their addresses
and the current stream, and calls the C ABI in ``libkvq.so``.  Every step of the computation
runs in the CUDA kernels; there is no CPU or PyTorch fallback.  If the library
has not been built, importing works but every call raises ``KvqError``.

Build: ``python -m kv_quant_cache_gb300._build`` (or ``__graft_entry__.build()``).
"""
from __future__ import annotations

import ctypes
import os

import torch

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG_DIR, "libkvq.so")

KVQ_OK = 0
KVQ_ERR_NULL = 1
KVQ_ERR_SHAPE = 2
KVQ_ERR_UNSUPPORTED = 3
KVQ_ERR_ALIGN = 4
KVQ_ERR_CUDA = 5
KVQ_ERR_VALUE = 6

ENTRY_BYTES = 584
DSV4_DIM = 512
DSV4_ROPE_DIM = 64  # rotated dims of a DSV4 row: cos/sin table width


class KvqError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(what)
        self.status = status


_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I = ctypes.c_int
_F = ctypes.c_float


def _declare(L: ctypes.CDLL) -> ctypes.CDLL:
    L.fused_qk_norm_rope.restype = _I
    L.fused_qk_norm_rope.argtypes = [_P, _I64, _I, _I, _I, _I, _F, _P, _P, _P, _I, _P, _P]
    L.fused_qk_norm_rope_ex.restype = _I
    L.fused_qk_norm_rope_ex.argtypes = [_P, _I64, _I, _I, _I, _I, _F, _P, _P, _P, _I, _I, _P,
                                        _P]
    L.dsv4_qnorm_rope_kv_rope_quant_insert.restype = _I
    L.dsv4_qnorm_rope_kv_rope_quant_insert.argtypes = [_P, _P, _I64, _I, _F, _P, _P, _P, _P,
                                                       _P, _P, _I, _P]
    L.dsv4_qnorm_rope_kv_rope_quant_insert_out.restype = _I
    L.dsv4_qnorm_rope_kv_rope_quant_insert_out.argtypes = [_P, _P, _P, _I64, _I, _F, _P, _P,
                                                           _P, _P, _P, _P, _I, _P]
    L.fused_qk_norm_rope_checked.restype = _I
    L.fused_qk_norm_rope_checked.argtypes = [_P, _I64, _I, _I, _I, _I, _F, _P, _P, _P, _I64, _I,
                                             _I, _P, _P, _P]
    L.dsv4_qnorm_rope_kv_rope_quant_insert_checked.restype = _I
    L.dsv4_qnorm_rope_kv_rope_quant_insert_checked.argtypes = [_P, _P, _P, _I64, _I, _F, _P, _P,
                                                               _P, _I64, _P, _P, _P, _I64, _I,
                                                               _P, _P]
    L.dsv4_kv_cache_gather_checked.restype = _I
    L.dsv4_kv_cache_gather_checked.argtypes = [_P, _I64, _I, _P, _I64, _P, _P, _P]
    L.dsv4_kv_cache_gather.restype = _I
    L.dsv4_kv_cache_gather.argtypes = [_P, _I, _P, _I64, _P, _P]
    L.paged_kv_rope_append.restype = _I
    L.paged_kv_rope_append.argtypes = [_P, _P, _I64, _I, _I, _I, _P, _I64, _I, _I, _P, _P, _P,
                                       _I64, _I, _P, _P]
    L.paged_kv_page_bounds.restype = _I
    L.paged_kv_page_bounds.argtypes = [_P, _I64, _I, _I, _I, _P, _P, _I64, _P, _P, _P]
    L.paged_kv_block_select.restype = _I
    L.paged_kv_block_select.argtypes = [_P, _I64, _I64, _I, _I, _I, _P, _I64, _I, _P, _I64, _I64,
                                        _P, _P, _I, _I, _I, _P, _P, _P]
    L.paged_block_sparse_attention_workspace.restype = _I64
    L.paged_block_sparse_attention_workspace.argtypes = [_I64, _I, _I, _I, _I, _I]
    L.paged_block_sparse_attention.restype = _I
    L.paged_block_sparse_attention.argtypes = [_P, _I64, _I64, _I, _I, _I, _P, _I64, _I, _P, _I64,
                                               _I64, _P, _P, _P, _I, _F, _P, _P, _I64, _P, _P]
    L.paged_shared_prefix_attention_workspace.restype = _I64
    L.paged_shared_prefix_attention_workspace.argtypes = [_I64, _I, _I, _I, _I, _I64, _I64]
    L.paged_shared_prefix_attention.restype = _I
    L.paged_shared_prefix_attention.argtypes = [_P, _I64, _I64, _I, _I, _I, _P, _I64, _I, _P, _I64,
                                                _P, _I64, _I64, _P, _P, _F, _P, _P, _I64, _P, _P]
    L.kvq_status_string.restype = ctypes.c_char_p
    L.kvq_status_string.argtypes = [_I]
    L.kvq_last_cuda_error.restype = _I
    L.kvq_last_cuda_error.argtypes = []
    L.kvq_dsv4_dispatch_threshold.restype = _I64
    L.kvq_dsv4_dispatch_threshold.argtypes = []
    L.kvq_set_dsv4_dispatch_threshold.restype = _I64
    L.kvq_set_dsv4_dispatch_threshold.argtypes = [_I64]
    L.kvq_dsv4_dispatch_path.restype = _I
    L.kvq_dsv4_dispatch_path.argtypes = [_I64, _I]
    for op in ("qk", "dsv4", "prefix"):
        getattr(L, f"kvq_{op}_num_configs").restype = _I
        getattr(L, f"kvq_{op}_num_configs").argtypes = []
        getattr(L, f"kvq_{op}_config_name").restype = ctypes.c_char_p
        getattr(L, f"kvq_{op}_config_name").argtypes = [_I]
        getattr(L, f"kvq_set_{op}_config").restype = _I
        getattr(L, f"kvq_set_{op}_config").argtypes = [_I]
    L.kvq_qk_config_for.restype = _I
    L.kvq_qk_config_for.argtypes = [_I64, _I, _I]
    L.kvq_set_stage_wait_limit.restype = ctypes.c_uint32
    L.kvq_set_stage_wait_limit.argtypes = [ctypes.c_uint32]
    L.kvq_set_tile_wait_limit.restype = ctypes.c_uint32
    L.kvq_set_tile_wait_limit.argtypes = [ctypes.c_uint32]
    L.kvq_stage_events.restype = _I
    L.kvq_stage_events.argtypes = [_P, _P, _I]
    L.kvq_set_programmatic_launch.restype = _I
    L.kvq_set_programmatic_launch.argtypes = [_I]
    L.kvq_dsv4_config_for.restype = _I
    L.kvq_dsv4_config_for.argtypes = [_I64, _I]
    return L


_LIB = None


def lib() -> ctypes.CDLL:
    """The loaded C library (raises KvqError if it has not been built)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise KvqError(-1, f"{LIB_PATH} not found: build it with "
                               "`python -m kv_quant_cache_gb300._build`")
        _LIB = _declare(ctypes.CDLL(LIB_PATH))
    return _LIB


def status_string(status: int) -> str:
    return lib().kvq_status_string(status).decode()


def _check(status: int, fn: str) -> None:
    if status != KVQ_OK:
        msg = f"{fn}: {status_string(status)}"
        if status == KVQ_ERR_CUDA:
            msg += f" (cudaError {lib().kvq_last_cuda_error()})"
        raise KvqError(status, msg)


def _cuda(t: torch.Tensor, dtype, name: str) -> int:
    """Address of a CUDA tensor, or of a pinned host tensor (mapped into the
    device's address space at the same address under unified addressing)."""
    if type(t) is torch.Tensor and t.is_cuda and t.dtype == dtype and t.is_contiguous():
        return t.data_ptr()  # the common case, checked first (per-call cost)
    # (a host tensor without elements counts as pinned: there is nothing to pin)
    if not isinstance(t, torch.Tensor) or not (t.is_cuda or (t.device.type == "cpu"
                                                             and (t.numel() == 0
                                                                  or t.is_pinned()))):
        raise ValueError(f"{name}: expected a CUDA tensor or a pinned host tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    return t.data_ptr()


# torch's current raw stream handle without building a Stream object (a few
# times cheaper per call); the public API is the fallback.
_raw_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, device) -> int:
    """Raw handle of ``stream`` (default: torch's current stream of ``device``,
    a CUDA device index; -1 = the current device)."""
    if stream is None:
        if _raw_current_stream is not None and device >= 0:
            return _raw_current_stream(device)
        stream = torch.cuda.current_stream(device if device >= 0 else None)
    if hasattr(stream, "cuda_stream"):
        sd = getattr(stream, "device", None)
        if device >= 0 and sd is not None and sd.index is not None and sd.index != device:
            raise ValueError(f"stream is on cuda:{sd.index}, the tensors on cuda:{device}")
        return stream.cuda_stream
    return int(stream)


# The current device as torch's runtime sees it (the raw query, without the
# public API's lazy-initialisation check; the public API is the fallback).
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _device(*tensors) -> int:
    """The one CUDA device that every CUDA tensor of a call is on (pinned host
    tensors, whose get_device() is -1, may take part on any device); -1 if
    none is a CUDA tensor."""
    dev = -1
    for t in tensors:
        if t is not None:
            d = t.get_device()
            if d != dev and d >= 0:
                if dev >= 0:
                    raise ValueError(f"tensors on cuda:{dev} and cuda:{d}: every CUDA tensor "
                                     "of one call must be on the same device")
                dev = d
    return dev


def _on(dev, fn, *args):
    """Call the C entry point ``fn`` with ``dev`` as the current device: the
    library launches on, and keeps its per-device set-up for, the current
    device, so a call whose tensors live on another GPU switches to it."""
    if dev >= 0 and dev != _current_device():
        with torch.cuda.device(dev):
            return fn(*args)
    return fn(*args)


def _counter(errors, name="errors"):
    return _cuda(errors, torch.int32, name)


def fused_qk_norm_rope(qkv, num_heads_q, num_heads_k, num_heads_v, head_dim, eps,
                       q_weight, k_weight, cos_sin_cache, is_neox, positions,
                       stream=None, rotary_dim=None, errors=None) -> None:
    """In-place per-head RMSNorm + RoPE of the Q and K heads of ``qkv``.

    qkv: bf16 [T, (Hq+Hk+Hv)*head_dim]; weights bf16 [head_dim]; cos_sin_cache
    fp32 [max_pos, rotary_dim]; positions int64 [T].  Same parameter order as
    the C entry point (stream last, default: torch's current stream).
    ``rotary_dim`` (default: the cos/sin table's width) selects partial
    rotation through ``fused_qk_norm_rope_ex``; ``is_neox`` picks NeoX (True)
    or GPT-J (False) pairs.  ``errors`` (an int32 CUDA tensor, zeroed by the
    caller) selects the bounds-checked launch: tokens whose position is
    outside the table are left unchanged and counted there.
    """
    if qkv.dim() != 2 or qkv.shape[1] != (num_heads_q + num_heads_k + num_heads_v) * head_dim:
        raise ValueError("qkv must be [T, (Hq+Hk+Hv)*head_dim]")
    if rotary_dim is None:
        rotary_dim = cos_sin_cache.shape[1]
    if cos_sin_cache.dim() != 2 or cos_sin_cache.shape[1] != rotary_dim:
        raise ValueError("cos_sin_cache must be [max_pos, rotary_dim]")
    T = qkv.shape[0]
    if q_weight.numel() != head_dim or k_weight.numel() != head_dim:
        raise ValueError("q_weight and k_weight must hold head_dim values")
    if positions.numel() != T:
        raise ValueError("positions must hold one value per token")
    dev = _device(qkv, q_weight, k_weight, cos_sin_cache, positions, errors)
    args = (_cuda(qkv, torch.bfloat16, "qkv"), T, num_heads_q, num_heads_k, num_heads_v,
            head_dim, float(eps), _cuda(q_weight, torch.bfloat16, "q_weight"),
            _cuda(k_weight, torch.bfloat16, "k_weight"),
            _cuda(cos_sin_cache, torch.float32, "cos_sin_cache"))
    tail = (int(rotary_dim), int(bool(is_neox)), _cuda(positions, torch.int64, "positions"))
    if errors is None:
        st = _on(dev, lib().fused_qk_norm_rope_ex, *args, *tail, _stream(stream, dev))
    else:
        st = _on(dev, lib().fused_qk_norm_rope_checked, *args, cos_sin_cache.shape[0], *tail,
                 _counter(errors), _stream(stream, dev))
    _check(st, "fused_qk_norm_rope")


def dsv4_qnorm_rope_kv_rope_quant_insert(q, kv, eps, q_weight, kv_weight, cos_sin_cache,
                                         positions, slot_mapping, kv_cache,
                                         stream=None, q_out=None, errors=None) -> None:
    """DSV4 prologue: q [T,H,512] normalised + rotated (in place, or into
    ``q_out`` when given); the kv vectors [T,512] normalised, rotated,
    quantised and written to ``kv_cache`` uint8 [num_blocks, block_size, 584]
    at ``slot_mapping``.  ``errors`` (int32 CUDA tensor, zeroed by the caller)
    selects the bounds-checked launch: tokens with a position outside the
    table or a slot outside the cache are rejected and counted there."""
    if q.dim() != 3 or q.shape[2] != DSV4_DIM:
        raise ValueError("q must be [T, H, 512]")
    if kv.dim() != 2 or kv.shape[0] != q.shape[0] or kv.shape[1] != DSV4_DIM:
        raise ValueError("kv must be [T, 512]")
    if kv_cache.dim() != 3 or kv_cache.shape[2] != ENTRY_BYTES:
        raise ValueError("kv_cache must be [num_blocks, block_size, 584]")
    T, H = q.shape[0], q.shape[1]
    if q_out is None:
        q_out = q
    if q_out.shape != q.shape:
        raise ValueError("q_out must have q's shape")
    if q_weight.numel() != DSV4_DIM or kv_weight.numel() != DSV4_DIM:
        raise ValueError("q_weight and kv_weight must hold 512 values")
    if cos_sin_cache.dim() != 2 or cos_sin_cache.shape[1] != DSV4_ROPE_DIM:
        raise ValueError("cos_sin_cache must be [max_pos, 64]")
    if positions.numel() != T or slot_mapping.numel() != T:
        raise ValueError("positions and slot_mapping must hold one value per token")
    dev = _device(q, q_out, kv, q_weight, kv_weight, cos_sin_cache, positions, slot_mapping,
                  kv_cache, errors)
    head = (_cuda(q, torch.bfloat16, "q"), _cuda(q_out, torch.bfloat16, "q_out"),
            _cuda(kv, torch.bfloat16, "kv"), T, H, float(eps),
            _cuda(q_weight, torch.bfloat16, "q_weight"),
            _cuda(kv_weight, torch.bfloat16, "kv_weight"),
            _cuda(cos_sin_cache, torch.float32, "cos_sin_cache"))
    idx = (_cuda(positions, torch.int64, "positions"),
           _cuda(slot_mapping, torch.int64, "slot_mapping"), _cuda(kv_cache, torch.uint8, "kv_cache"))
    if errors is None:
        st = _on(dev, lib().dsv4_qnorm_rope_kv_rope_quant_insert_out, *head, *idx,
                 kv_cache.shape[1], _stream(stream, dev))
    else:
        st = _on(dev, lib().dsv4_qnorm_rope_kv_rope_quant_insert_checked,
                 *head, cos_sin_cache.shape[0], *idx, kv_cache.shape[0], kv_cache.shape[1],
                 _counter(errors), _stream(stream, dev))
    _check(st, "dsv4_qnorm_rope_kv_rope_quant_insert")


def dsv4_kv_cache_gather(kv_cache, slots, out=None, stream=None, errors=None):
    """bf16 [n, 512] rows read back from the cache entries at ``slots``
    (int64 [n], -1 = a zero row); ``out`` is allocated if not given.
    ``errors`` (int32 CUDA tensor) selects the bounds-checked launch."""
    if kv_cache.dim() != 3 or kv_cache.shape[2] != ENTRY_BYTES:
        raise ValueError("kv_cache must be [num_blocks, block_size, 584]")
    if slots.dim() != 1:
        raise ValueError("slots must be a 1-D int64 tensor")
    n = slots.shape[0]
    if out is None:
        out = torch.empty((n, DSV4_DIM), dtype=torch.bfloat16, device=kv_cache.device)
    if out.shape != (n, DSV4_DIM):
        raise ValueError("out must be [len(slots), 512]")
    dev = _device(kv_cache, slots, out, errors)
    if errors is None:
        st = _on(dev, lib().dsv4_kv_cache_gather,
                 _cuda(kv_cache, torch.uint8, "kv_cache"), kv_cache.shape[1],
                 _cuda(slots, torch.int64, "slots"), n, _cuda(out, torch.bfloat16, "out"),
                 _stream(stream, dev))
    else:
        st = _on(dev, lib().dsv4_kv_cache_gather_checked,
                 _cuda(kv_cache, torch.uint8, "kv_cache"), kv_cache.shape[0], kv_cache.shape[1],
                 _cuda(slots, torch.int64, "slots"), n, _cuda(out, torch.bfloat16, "out"),
                 _counter(errors), _stream(stream, dev))
    _check(st, "dsv4_kv_cache_gather")
    return out


# ---- paged grouped-query operators ---------------------------------------------------
# A decode step calls each of these once a layer, and for small batches the
# call costs the host more than the kernel costs the GPU, so their argument
# checks are written for few interpreter steps: one helper call per tensor,
# sizes unpacked once, workspace sizes (a function of the sizes alone)
# remembered.

_BF16, _I32, _I64T, _F32 = torch.bfloat16, torch.int32, torch.int64, torch.float32


def _ptr(t, dtype, dev, name) -> int:
    """Address of a contiguous ``dtype`` tensor on CUDA device ``dev`` (or of a
    pinned host tensor, which may take part on any device)."""
    if t.dtype is dtype and t.is_contiguous() and t.get_device() == dev:
        if dev >= 0:
            return t.data_ptr()
    ptr = _cuda(t, dtype, name)
    if t.get_device() not in (dev, -1):
        raise ValueError(f"{name}: on cuda:{t.get_device()}, other tensors of the call on "
                         f"cuda:{dev}: every CUDA tensor of one call must be on the same device")
    return ptr


def _home(t, *others) -> int:
    """The CUDA device of a call: that of ``t``, or, where ``t`` is a pinned
    host tensor, of the first CUDA tensor among the others (-1: there is
    none)."""
    dev = t.get_device()
    return dev if dev >= 0 else _device(*others)


def _launch(dev, stream, fn, *args) -> None:
    """``fn(*args, stream)`` on device ``dev``; raises on an error status."""
    if dev >= 0 and dev != _current_device():
        with torch.cuda.device(dev):
            st = fn(*args, _stream(stream, dev))
    else:
        st = fn(*args, _stream(stream, dev))
    if st:
        _check(st, fn.__name__)


_DEVICES = {}


def _new(shape, dtype, dev, stream):
    """An output or workspace on the call's device, allocated for the stream of
    the call: memory that other streams still use is not given to it, nor its
    memory to them when it is freed.  Where every tensor of the call is pinned
    host memory so is an output; that has no order of streams, and like the
    call's other tensors it is the caller's to keep until the call is done."""
    if dev >= 0:
        where = _DEVICES.get(dev)
        if where is None:  # building a device object costs more than the look-up
            where = _DEVICES[dev] = torch.device("cuda", dev)
        if stream is None:
            return torch.empty(shape, dtype=dtype, device=where)
        handle = _stream(stream, dev)
        of_call = (torch.cuda.ExternalStream(handle, device=where) if handle
                   else torch.cuda.default_stream(where))
        with torch.cuda.stream(of_call):
            return torch.empty(shape, dtype=dtype, device=where)
    return torch.empty(shape, dtype=dtype, pin_memory=True)


def _counted(errors, dev):
    return None if errors is None else _ptr(errors, _I32, dev, "errors")


def _paged_cache(kv_cache):
    """num_pages, Hkv, page_size, head_dim of a paged cache."""
    if kv_cache.dim() == 5:
        pages, two, heads, page, dim = kv_cache.shape
        if two == 2:
            return pages, heads, page, dim
    raise ValueError("kv_cache must be [num_pages, 2, Hkv, page_size, head_dim]")


def paged_kv_rope_append(qkv, num_heads_q, num_heads_kv, head_dim, cos_sin_cache, is_neox,
                         positions, slot_mapping, kv_cache, q_out=None, stream=None,
                         rotary_dim=None, errors=None) -> None:
    """RoPE of the Q and K heads of ``qkv`` [T, (Hq+2Hkv)*head_dim] and the K
    and V heads written to ``kv_cache`` (bf16 [num_pages, 2, Hkv, page_size,
    head_dim]) at ``slot_mapping`` (int64 [T], -1 = none), in one pass.  The
    rotated query rows go to ``q_out`` (bf16 [T, Hq, head_dim]) or stay in
    place.  ``cos_sin_cache`` None: no rotation (after fused_qk_norm_rope);
    ``rotary_dim`` defaults to the table's width.  Tokens with a position
    outside the table are left out, slots outside the cache not written; both
    are counted in ``errors`` (int32 CUDA tensor) when given."""
    pages, heads, page, dim = _paged_cache(kv_cache)
    if heads != num_heads_kv or dim != head_dim:
        raise ValueError("kv_cache must be [num_pages, 2, Hkv, page_size, head_dim] of the "
                         "call's Hkv and head_dim")
    if qkv.dim() != 2 or qkv.shape[1] != (num_heads_q + 2 * num_heads_kv) * head_dim:
        raise ValueError("qkv must be [T, (Hq+2*Hkv)*head_dim]")
    T = qkv.shape[0]
    if slot_mapping.numel() != T:
        raise ValueError("slot_mapping must hold one value per token")
    dev = _home(qkv, q_out, cos_sin_cache, positions, slot_mapping, kv_cache, errors)
    q_ptr = None
    if q_out is not None:
        if q_out.shape != (T, num_heads_q, head_dim):
            raise ValueError("q_out must be [T, Hq, head_dim]")
        q_ptr = _ptr(q_out, _BF16, dev, "q_out")
    if cos_sin_cache is None:
        if rotary_dim:
            raise ValueError("rotary_dim without a cos_sin_cache")
        rows = rot = 0
        cs = pos = None
    else:
        rows, rot = cos_sin_cache.shape if cos_sin_cache.dim() == 2 else (0, 0)
        if rot == 0 or (rotary_dim is not None and rotary_dim != rot):
            raise ValueError("cos_sin_cache must be [max_pos, rotary_dim]")
        if positions.numel() != T:
            raise ValueError("positions must hold one value per token")
        cs = _ptr(cos_sin_cache, _F32, dev, "cos_sin_cache")
        pos = _ptr(positions, _I64T, dev, "positions")
    _launch(dev, stream, (_LIB or lib()).paged_kv_rope_append, _ptr(qkv, _BF16, dev, "qkv"), q_ptr,
            T, num_heads_q, num_heads_kv, head_dim, cs, rows, rot, 1 if is_neox else 0, pos,
            _ptr(slot_mapping, _I64T, dev, "slot_mapping"),
            _ptr(kv_cache, _BF16, dev, "kv_cache"), pages, page, _counted(errors, dev))


def paged_kv_page_bounds(kv_cache, pages, lens, bounds, stream=None, errors=None):
    """Writes the smallest and largest key per dim of the first ``lens``
    (int32 [n]) tokens of each listed page (int64 [n], -1 = none) into
    ``bounds`` (bf16 [num_pages, Hkv, 2, head_dim]), and returns ``bounds``."""
    N, Hkv, page, D = _paged_cache(kv_cache)
    if pages.dim() != 1 or lens.shape != pages.shape:
        raise ValueError("pages and lens must be 1-D, of one length")
    if bounds.shape != (N, Hkv, 2, D):
        raise ValueError("bounds must be [num_pages, Hkv, 2, head_dim]")
    dev = _home(kv_cache, pages, lens, bounds, errors)
    _launch(dev, stream, (_LIB or lib()).paged_kv_page_bounds,
            _ptr(kv_cache, _BF16, dev, "kv_cache"), N, Hkv, page, D,
            _ptr(pages, _I64T, dev, "pages"), _ptr(lens, _I32, dev, "lens"), pages.shape[0],
            _ptr(bounds, _BF16, dev, "bounds"), _counted(errors, dev))
    return bounds


def _paged_q(q, head_dim, dev):
    """Address, tokens, heads and token stride of bf16 [T, Hq, D] whose heads
    are contiguous (a token's rows may be a view into packed QKV)."""
    if q.dim() != 3:
        raise ValueError(f"q must be [T, Hq, {head_dim}]")
    T, Hq, D = q.shape
    if D != head_dim:
        raise ValueError(f"q must be [T, Hq, {head_dim}]")
    if q.dtype is not _BF16:
        raise ValueError(f"q: expected {_BF16}, got {q.dtype}")
    if dev < 0 or q.get_device() != dev:
        if not (q.is_cuda or (q.device.type == "cpu" and (q.numel() == 0 or q.is_pinned()))):
            raise ValueError("q: expected a CUDA tensor or a pinned host tensor")
    if q.is_contiguous() or T == 0:
        return q.data_ptr(), T, Hq, Hq * D
    st, sh, sd = q.stride()
    if sd != 1 or (Hq > 1 and sh != D):
        raise ValueError("q: the heads of a token must be contiguous")
    return q.data_ptr(), T, Hq, (st if T > 1 else Hq * D)


def _requests(T, page_table, lens, requests):
    """num_requests and table_width of a call with T tokens."""
    if page_table.dim() != 2:
        raise ValueError("page_table must be [num_requests, table_width]")
    R, width = page_table.shape
    if lens.numel() != T or (requests is not None and requests.numel() != T):
        raise ValueError("lens and requests must hold one value per token")
    if requests is None and R < T:
        raise ValueError("page_table must have a row per token when requests is not given")
    return R, width


def paged_kv_block_select(q, bounds, page_table, lens, page_size, topk, keep_first=0,
                          keep_last=0, out=None, requests=None, stream=None, errors=None):
    """int32 [T, Hkv, topk]: for each token of ``q`` [T, Hq, D] and kv head the
    blocks (pages of the token's request) with the highest scores from
    ``bounds`` (paged_kv_page_bounds), ascending, then -1.  ``page_table``
    int32 [requests, width]; ``lens`` int32 [T]: keys each token sees;
    ``requests`` int32 [T] (default: token t is request t); ``keep_first`` /
    ``keep_last`` blocks are always selected."""
    if bounds.dim() != 4 or bounds.shape[2] != 2:
        raise ValueError("bounds must be [num_pages, Hkv, 2, head_dim]")
    N, Hkv, _, D = bounds.shape
    dev = _home(q, bounds, page_table, lens, requests, out, errors)
    q_ptr, T, Hq, q_stride = _paged_q(q, D, dev)
    R, width = _requests(T, page_table, lens, requests)
    if out is None:
        out = _new((T, Hkv, topk), _I32, dev, stream)
    elif out.shape != (T, Hkv, topk):
        raise ValueError("out must be [T, Hkv, topk]")
    _launch(dev, stream, (_LIB or lib()).paged_kv_block_select, q_ptr, q_stride, T, Hq, Hkv, D,
            _ptr(bounds, _BF16, dev, "bounds"), N, page_size,
            _ptr(page_table, _I32, dev, "page_table"), R, width,
            None if requests is None else _ptr(requests, _I32, dev, "requests"),
            _ptr(lens, _I32, dev, "lens"), topk, keep_first, keep_last,
            _ptr(out, _I32, dev, "out"), _counted(errors, dev))
    return out


# Sizes of a call -> bytes of workspace it needs.  set_config puts an empty table
# in its place: what another thread found under the setting before goes into the
# old one.
_WORKSPACE = {}


def _workspace_bytes(fn, *sizes) -> int:
    table = _WORKSPACE
    need = table.get((fn, sizes))
    if need is None:
        if len(table) >= 4096:
            table.clear()
        need = table[(fn, sizes)] = getattr(lib(), fn)(*sizes)
    return need


def _output(q, out, dev, stream):
    if out is None:
        return _new(q.shape, _BF16, dev, stream)
    if out.shape != q.shape:
        raise ValueError("out must have q's shape")
    return out


# Memory of torch's allocator without a tensor around it, on the current device
# for a stream (after a launch a tensor costs 4 us to make, this 1 us).
_raw_alloc = getattr(torch._C, "_cuda_cudaCachingAllocator_raw_alloc", None)
_raw_free = getattr(torch._C, "_cuda_cudaCachingAllocator_raw_delete", None)


def _launch_attention(dev, stream, fn, args, workspace, need, errors) -> None:
    """``fn(*args, workspace, its bytes, errors, stream)``.  A workspace of
    ``need`` bytes that is not given is allocated for the call alone: torch's
    allocator hands it on in the order of the call's stream.  It is device
    memory for pinned tensors too: given back, pinned memory would be handed on
    at once, with the call's kernels still to write it."""
    errors = _counted(errors, dev)
    here = dev if dev >= 0 or not need else _current_device()
    if workspace is None and need and _raw_free and here == _current_device():
        handle = _stream(stream, dev)
        ws = _raw_alloc(need, handle)
        try:
            st = fn(*args, ws, need, errors, handle)
        finally:
            _raw_free(ws)
        if st:
            _check(st, fn.__name__)
        return
    if workspace is None:
        workspace = _new(need, torch.uint8, here, stream) if need else None
        _launch(dev, stream, fn, *args, workspace.data_ptr() if need else None, need, errors)
    else:
        _launch(dev, stream, fn, *args, _ptr(workspace, workspace.dtype, dev, "workspace"),
                workspace.numel() * workspace.element_size(), errors)


def paged_block_sparse_attention(q, kv_cache, page_table, blocks, lens, scale=None, out=None,
                                 requests=None, workspace=None, stream=None, errors=None):
    """bf16 [T, Hq, D]: attention of each token of ``q`` over the keys of the
    cache blocks listed for it (``blocks`` int32 [T, Hkv, topk], -1 = none, as
    paged_kv_block_select returns them) that lie below ``lens[t]``.  ``scale``
    defaults to 1/sqrt(D).  ``workspace``: a tensor of at least
    ``paged_block_sparse_attention_workspace`` bytes, allocated per call if
    needed and not given."""
    N, Hkv, page, D = _paged_cache(kv_cache)
    dev = _home(q, kv_cache, page_table, blocks, lens, requests, out, errors, workspace)
    q_ptr, T, Hq, q_stride = _paged_q(q, D, dev)
    B, H, topk = blocks.shape if blocks.dim() == 3 else (-1, 0, 0)
    if B != T or H != Hkv:
        raise ValueError("blocks must be [T, Hkv, topk]")
    R, width = _requests(T, page_table, lens, requests)
    out = _output(q, out, dev, stream)
    need = _workspace_bytes("paged_block_sparse_attention_workspace", T, Hq, Hkv, D, page, topk)
    _launch_attention(
        dev, stream, (_LIB or lib()).paged_block_sparse_attention,
        (q_ptr, q_stride, T, Hq, Hkv, D, _ptr(kv_cache, _BF16, dev, "kv_cache"), N, page,
         _ptr(page_table, _I32, dev, "page_table"), R, width,
         None if requests is None else _ptr(requests, _I32, dev, "requests"),
         _ptr(lens, _I32, dev, "lens"), _ptr(blocks, _I32, dev, "blocks"), topk,
         D ** -0.5 if scale is None else scale, _ptr(out, _BF16, dev, "out")),
        workspace, need, errors)
    return out


def paged_shared_prefix_attention(q, kv_cache, prefix_pages, prefix_len, page_table, lens,
                                  scale=None, out=None, requests=None, workspace=None,
                                  stream=None, errors=None):
    """bf16 [T, Hq, D]: attention of each token of ``q`` over the shared
    ``prefix_len`` keys of ``prefix_pages`` (int32) and the first ``lens[t]``
    keys of its own request's pages (``page_table``).  The prefix is read once
    for the whole batch.  Other arguments as paged_block_sparse_attention."""
    N, Hkv, page, D = _paged_cache(kv_cache)
    dev = _home(q, kv_cache, prefix_pages, page_table, lens, requests, out, errors, workspace)
    q_ptr, T, Hq, q_stride = _paged_q(q, D, dev)
    if prefix_pages.dim() != 1 or prefix_pages.shape[0] * page < prefix_len:
        raise ValueError("prefix_pages must be 1-D and hold prefix_len keys")
    R, width = _requests(T, page_table, lens, requests)
    out = _output(q, out, dev, stream)
    need = _workspace_bytes("paged_shared_prefix_attention_workspace", T, Hq, Hkv, D, page,
                            prefix_len, width)
    _launch_attention(
        dev, stream, (_LIB or lib()).paged_shared_prefix_attention,
        (q_ptr, q_stride, T, Hq, Hkv, D, _ptr(kv_cache, _BF16, dev, "kv_cache"), N, page,
         _ptr(prefix_pages, _I32, dev, "prefix_pages"), prefix_len,
         _ptr(page_table, _I32, dev, "page_table"), R, width,
         None if requests is None else _ptr(requests, _I32, dev, "requests"),
         _ptr(lens, _I32, dev, "lens"), D ** -0.5 if scale is None else scale,
         _ptr(out, _BF16, dev, "out")), workspace, need, errors)
    return out


def dsv4_dispatch_threshold() -> int:
    return lib().kvq_dsv4_dispatch_threshold()


def set_dsv4_dispatch_threshold(value: int) -> int:
    """Set the DSV4 program-count threshold (< 0 restores the default); returns the old one."""
    return lib().kvq_set_dsv4_dispatch_threshold(int(value))


def dsv4_dispatch_path(num_tokens: int, num_heads: int) -> int:
    return lib().kvq_dsv4_dispatch_path(int(num_tokens), int(num_heads))


def configs(op: str) -> list:
    """Names of the launch configurations of ``op`` ("qk", "dsv4" or "prefix")."""
    L = lib()
    n = getattr(L, f"kvq_{op}_num_configs")()
    return [getattr(L, f"kvq_{op}_config_name")(i).decode() for i in range(n)]


def set_config(op: str, config_id: int) -> int:
    """Force launch configuration ``config_id`` of ``op`` (< 0: automatic);
    returns the previous override."""
    prev = getattr(lib(), f"kvq_set_{op}_config")(int(config_id))
    if prev == -2:
        raise ValueError(f"{op}: no launch configuration {config_id}")
    global _WORKSPACE
    _WORKSPACE = {}  # what a call needs may depend on it
    return prev


def set_stage_wait_limit(polls: int) -> int:
    """Polls of a stage barrier before a warp of a staged QK launch shape
    finishes from global memory (0: always); returns the previous limit."""
    return lib().kvq_set_stage_wait_limit(int(polls))


def set_tile_wait_limit(polls: int) -> int:
    """Polls of a barrier before a CTA of the shared prefix's tensor-core tiles
    gives up, and its rows become NaN (0: without a poll); returns the previous
    limit."""
    return lib().kvq_set_tile_wait_limit(int(polls))


def stage_events(reset: bool = False) -> tuple:
    """(fallbacks, drain_timeouts) counted by the staged QK launch shapes on
    the current device since the last reset (waits for the device first)."""
    fb, dt = ctypes.c_uint64(0), ctypes.c_uint64(0)
    _check(lib().kvq_stage_events(ctypes.addressof(fb), ctypes.addressof(dt), int(bool(reset))),
           "kvq_stage_events")
    return fb.value, dt.value


def set_programmatic_launch(enable: bool) -> bool:
    """Launch later kernels with programmatic stream serialization (the
    default: they may be scheduled while the previous kernel finishes; results
    are unchanged); returns the previous setting."""
    return bool(lib().kvq_set_programmatic_launch(1 if enable else 0))


def qk_config_for(num_tokens: int, num_heads_q: int, num_heads_k: int) -> int:
    return lib().kvq_qk_config_for(int(num_tokens), int(num_heads_q), int(num_heads_k))


def dsv4_config_for(num_tokens: int, num_heads: int) -> int:
    return lib().kvq_dsv4_config_for(int(num_tokens), int(num_heads))
