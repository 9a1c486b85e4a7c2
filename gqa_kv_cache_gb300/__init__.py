"""GQA decode step over a KV cache on GB300 (sm_103a).

Thin Python binding of ``libgqa.so``: it checks tensor shapes and dtypes,
passes device pointers and the current CUDA stream to the C ABI
(include/gqa_decode.h) and raises on error codes. Every step of the decode
runs in the library's CUDA kernels; PyTorch only provides device memory and
streams. There is no CPU fallback: without the built library or a GPU the
calls raise.

One decode step, per batch row b: the new key/value are appended in place at
slot ``lengths[b]`` of the row's cache, and every query head h attends over
slots ``0..lengths[b]`` of cache head ``h // (Hq // Hkv)`` with a float32
softmax of ``q.K/sqrt(D)``; the output is float32 (B, Hq, D).

The read-only attend (``attend``, ``attend_paged``) attends slots
``0..lengths[b]-1`` (lengths counts the valid slots) and writes nothing but
its output; its query may be float32 over a bfloat16 cache.

A cache of E4M3 (FP8) bytes (``torch.uint8`` or ``torch.float8_e4m3fn``
tensors) takes ``k_scale`` / ``v_scale`` float32 (Hkv,) tensors: K =
k_scale[kvh] * K8; the decode step then takes bfloat16 q, k_new and v_new and
quantises the appended token.

A cache of 4-bit E2M1 values holds D / 2 bytes a vector (``torch.uint8`` or
``torch.float4_e2m1fn_x2``) and takes ``k_group_scale`` / ``v_group_scale``
besides: E4M3 bytes of the cache's shape with D // 16 last, one scale per 16
dims (the format is the C header's GQA_DTYPE_E2M1).

``append`` and ``append_paged`` write packed tokens into any of these caches
without attending (and keep the key bounds of its blocks), ``read`` and
``read_paged`` give slots back as vectors. ``select_blocks`` and
``select_blocks_paged`` choose the blocks of slots whose key bounds promise
the highest scores, and ``attend_selected`` attends those alone.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import _lib

__all__ = ["decode_step", "decode_step_paged", "attend", "attend_paged", "decode_multi",
           "decode_multi_paged", "append", "append_paged", "read", "read_paged", "select_blocks",
           "select_blocks_paged", "attend_selected", "Selection", "workspace_bytes", "validate", "validate_attend", "validate_multi",
           "GqaError", "trace_enable", "trace_collect", "KERNELS", "library_path"]

OK, INVALID_ARGUMENT, UNSUPPORTED, CUDA_ERROR, WORKSPACE = 0, 1, 2, 3, 4
KERNELS = {"auto": 0, "simt": 1, "tc": 2, "unit": 3, "tc5": 4}
STATUS_BITS = {1: "bad length", 2: "bad slot id", 4: "bad block", 8: "timeout", 16: "bad kept prefix",
               32: "bad token offsets"}
_DTYPES = {torch.float32: 0, torch.bfloat16: 1}
E4M3, E2M1 = 2, 3
_GROUP = 16   # dims that share an E4M3 scale in an E2M1 cache
_NIBBLE_DTYPES = (torch.uint8,) + ((torch.float4_e2m1fn_x2,) if hasattr(torch, "float4_e2m1fn_x2") else ())
_BYTE_DTYPES = (torch.uint8,) + ((torch.float8_e4m3fn,) if hasattr(torch, "float8_e4m3fn") else ())


def _cache_code(t) -> int:
    """gqa_dtype of a cache tensor."""
    if t.dtype in _BYTE_DTYPES:
        return E4M3
    if t.dtype not in _DTYPES:
        raise TypeError("a cache must be float32, bfloat16 or E4M3 bytes")
    return _DTYPES[t.dtype]

library_path = _lib.LIB_PATH


class GqaError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        msg = _lib.load().gqa_status_string(code).decode()
        super().__init__(f"{what}: {msg} (status {code})")


def _check(code: int, what: str):
    if code != OK:
        raise GqaError(code, what)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _head_scale(name, t, Hkv, device):
    if t.dtype != torch.float32 or t.shape != (Hkv,) or not t.is_contiguous() or t.get_device() != device.index:
        raise TypeError(f"{name} must be a contiguous float32 (Hkv,) tensor on q's device")
    return t.data_ptr()


def _opts(kernel, grid_ctas, sched_pad=None, sink=None, window=0, kept_prefix=0, device=None, B=None,
          Hq=None, k_scale=None, v_scale=None, Hkv=None, wait_limit_cycles=0, test_stall=False,
          k_group_scale=None, v_group_scale=None):
    """The gqa_options struct. Softmax modifiers: ``sink`` a float32 (Hq,)
    device tensor, ``window`` an int >= 0, ``kept_prefix`` an int >= 0 or an
    int32 (B,) device tensor. ``wait_limit_cycles`` > 0 shortens the
    tensor-core consumers' wait for a tile to that many SM clock cycles and
    ``test_stall`` makes each consumer's first wait one that runs out (both
    for tests of the timeout path)."""
    o = _lib.GqaOptions()   # zeros: the defaults (a field is set only where it differs: setting costs time)
    if wait_limit_cycles:
        o.wait_limit_cycles = int(wait_limit_cycles)
    if test_stall:
        o.test_stall = 1
    if kernel != "auto":
        o.kernel = KERNELS[kernel] if isinstance(kernel, str) else int(kernel)
    if grid_ctas:
        o.grid_ctas = int(grid_ctas)
    if sched_pad is not None:
        o.sched_pad = int(sched_pad) + 1   # 0 = library default
    if window:
        o.window = int(window)
    if sink is not None:
        if sink.dtype != torch.float32 or sink.shape != (Hq,) or not sink.is_contiguous() \
                or sink.device != device:
            raise TypeError("sink must be a contiguous float32 (Hq,) tensor on q's device")
        o.head_sink = sink.data_ptr()
    if isinstance(kept_prefix, torch.Tensor):
        if kept_prefix.dtype != torch.int32 or kept_prefix.shape != (B,) \
                or not kept_prefix.is_contiguous() or kept_prefix.device != device:
            raise TypeError("kept_prefix must be an int or a contiguous int32 (B,) tensor on q's device")
        o.kept_prefix_rows = kept_prefix.data_ptr()
    elif kept_prefix:
        o.kept_prefix = int(kept_prefix)
    if k_scale is not None:
        o.k_scale = _head_scale("k_scale", k_scale, Hkv, device)
    if v_scale is not None:
        o.v_scale = _head_scale("v_scale", v_scale, Hkv, device)
    if k_group_scale is not None:
        o.k_group_scale = k_group_scale.data_ptr()
        o.v_group_scale = v_group_scale.data_ptr()
    return o


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)   # current_stream without its Python object


def _stream(stream, device=None):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device() if device is None else device.index)
    return torch.cuda.current_stream(device).cuda_stream


_ws_cache: dict = {}
_ws_captured: dict = {}   # (capture, workspace) of the captures under way, by stream


def _workspace(device, nbytes, stream=None):
    """A workspace of the device and stream, zero-filled when allocated; the
    library leaves it zero-filled after every call, whatever the sizes. Calls
    on one stream run one after the other; each stream has its own, and so has
    each stream of a capture (the graph fills it with zeros before its first
    call, and may then be replayed beside any other work)."""
    handle = _stream(stream, device)
    capture = 0
    if stream is not None or torch.cuda.is_current_stream_capturing():
        n = ctypes.c_uint64()
        _check(_lib.load().gqa_stream_capture_id(handle, ctypes.byref(n)), "gqa_stream_capture_id")
        capture = n.value
    key = (device, handle) if handle else device
    if capture:
        was, buf = _ws_captured.get(key, (0, None))
        if was == capture and buf.numel() >= nbytes:
            return buf
    else:
        if _ws_captured:   # the graphs' own memory is theirs once their captures are over
            _ws_captured.clear()
        buf = _ws_cache.get(key)
        if buf is not None and buf.numel() >= nbytes:
            return buf
    with torch.cuda.stream(stream) if stream is not None else _HERE:   # zero-filled before the stream's next kernel
        buf = torch.zeros(max(nbytes, 1 if capture else 1 << 20), dtype=torch.uint8, device=device)
    if capture:
        _ws_captured[key] = capture, buf
    else:
        _ws_cache[key] = buf
    return buf


_need_cache: dict = {}


def _need(lib, B, Hq, Hkv, D, dt, kernel, grid_ctas, o, device):
    """gqa_workspace_bytes of these sizes on this device (asked once)."""
    key = (B, Hq, Hkv, D, dt, kernel, grid_ctas, device.index)
    n = _need_cache.get(key)
    if n is None:
        n = _need_cache[key] = lib.gqa_workspace_bytes(B, Hq, Hkv, D, dt, ctypes.byref(o))
    return n


def _on(device):
    """The device as the current one, where it is not."""
    if device.index == torch.cuda.current_device():
        return _HERE
    return torch.cuda.device(device)


_HERE = contextlib.nullcontext()


def workspace_bytes(B, Hq, Hkv, D, dtype=torch.bfloat16, kernel="auto", grid_ctas=0) -> int:
    """Workspace bytes the library needs for one step of these sizes.
    ``dtype`` is the cache's; "e2m1" for a 4-bit cache."""
    o = _opts(kernel, grid_ctas)
    code = E2M1 if dtype == "e2m1" else E4M3 if dtype in _BYTE_DTYPES else _DTYPES[dtype]
    return int(_lib.load().gqa_workspace_bytes(B, Hq, Hkv, D, code, ctypes.byref(o)))


def _group_scales(caches, k_group_scale, v_group_scale, D):
    """Checks of an E2M1 cache's tensors (the shapes against D dims a vector)."""
    (kname, k), (vname, v) = caches
    if k.dtype not in _NIBBLE_DTYPES or v.dtype not in _NIBBLE_DTYPES:
        raise TypeError(f"{kname} and {vname} with group scales must hold E2M1 pairs (uint8 or float4_e2m1fn_x2)")
    if k_group_scale is None or v_group_scale is None or k_group_scale.dtype not in _BYTE_DTYPES \
            or v_group_scale.dtype not in _BYTE_DTYPES:
        raise TypeError("k_group_scale and v_group_scale must both be E4M3 bytes (uint8 or float8_e4m3fn)")
    shape = k.shape
    groups = (*shape[:-1], D // _GROUP)
    if D % _GROUP or shape[-1] * 2 != D or v.shape != shape or k_group_scale.shape != groups \
            or v_group_scale.shape != groups:
        raise ValueError(f"{kname} and {vname} must hold D // 2 bytes a vector and the group scales D // {_GROUP}, D = {D}")
    dev = k.get_device()
    if k_group_scale.get_device() != dev or v_group_scale.get_device() != dev \
            or not k_group_scale.is_contiguous() or not v_group_scale.is_contiguous():
        raise ValueError("the group scales must be contiguous and on the caches' device")


def _plain(dev, *tensors):
    """Raises unless every tensor given is contiguous and on device `dev`."""
    for t in tensors:
        if t is not None and (t.get_device() != dev or not t.is_contiguous()):
            raise ValueError("every tensor must be contiguous and on q's device")


def _check_e2m1(q, k, v, kg, vg, out):
    """Checks of a query, a 4-bit cache and an output that was given; returns the device index."""
    dev = q.get_device()
    if dev < 0:
        raise ValueError("tensors must be on a CUDA device")
    if q.dtype not in _DTYPES:
        raise TypeError("q must be float32 or bfloat16")
    _group_scales((("the key cache", k), ("the value cache", v)), kg, vg, q.shape[2])
    _plain(dev, q, k, v, out)
    if out is not None and (out.shape != q.shape or out.dtype != torch.float32):
        raise ValueError("out must be a contiguous float32 (B, Hq, D) tensor on q's device")
    return dev


def _step_e2m1(q, k_new, v_new, k, v, lengths, slot_ids, table, k_scale, v_scale, kg, vg, out, status, kernel,
               grid_ctas, workspace, stream, sched_pad, sink, window, kept_prefix):
    """The decode step (k_new, v_new given) or the attend over a 4-bit cache,
    dense or paged (table given). Written out for itself: the step is short,
    and its time on the host counts."""
    dev = _check_e2m1(q, k, v, kg, vg, out)
    B, Hq, D = q.shape
    n0, Hkv, n2, _ = k.shape
    if Hq % Hkv or lengths.shape != (B,):
        raise ValueError("shape mismatch between q, the caches and lengths")
    if lengths.dtype != torch.int32:
        raise TypeError("lengths must be a contiguous int32 tensor on q's device")
    if slot_ids is not None and (slot_ids.dtype != torch.int32 or slot_ids.shape != (B,)):
        raise TypeError("slot_ids must be int32 of shape (B,)")
    if table is not None and (table.dtype != torch.int32 or table.dim() != 2 or table.shape[0] != B):
        raise TypeError("block_table must be a contiguous int32 (B, max_blocks) tensor")
    _plain(dev, lengths, slot_ids, table, k_new, v_new)
    if k_new is not None:
        if q.dtype != torch.bfloat16 or k_new.dtype != torch.bfloat16 or v_new.dtype != torch.bfloat16:
            raise TypeError("over an E2M1 cache q, k_new and v_new are bfloat16")
        if k_new.shape != (B, Hkv, D) or v_new.shape != (B, Hkv, D):
            raise ValueError("shape mismatch between q, k_new and v_new")
    device = q.device
    if status is not None:
        _status_checks(status, device)
    if workspace is not None:
        _plain(dev, workspace)
    o = _opts(kernel, grid_ctas, sched_pad, sink, window, kept_prefix, device, B, Hq, k_scale, v_scale, Hkv,
              k_group_scale=kg, v_group_scale=vg)
    lib = _lib.load()
    if stream is not None and out is None:   # the memory of the stream that writes it
        with torch.cuda.stream(stream):
            out = torch.empty(q.shape, dtype=torch.float32, device=device)
    with _on(device):
        need = _need(lib, B, Hq, Hkv, D, E2M1, kernel, grid_ctas, o, device)
        ws = _workspace(device, need, stream) if workspace is None else workspace
        at, size, st = ws.data_ptr(), ws.numel() * ws.element_size(), _ptr(status)
        if out is None:   # last: right after another launch an allocation takes longer (4.6 us for 1.4)
            out = torch.empty_like(q, dtype=torch.float32)
        if table is None:
            if k_new is None:
                what, code = "gqa_attend", lib.gqa_attend(
                    q.data_ptr(), _DTYPES[q.dtype], k.data_ptr(), v.data_ptr(), lengths.data_ptr(), _ptr(slot_ids),
                    out.data_ptr(), B, Hq, Hkv, D, n0, n2, E2M1, at, size, st, _stream(stream), ctypes.byref(o))
            else:
                what, code = "gqa_decode_step", lib.gqa_decode_step_ex(
                    q.data_ptr(), k_new.data_ptr(), v_new.data_ptr(), k.data_ptr(), v.data_ptr(), lengths.data_ptr(),
                    _ptr(slot_ids), out.data_ptr(), B, Hq, Hkv, D, n0, n2, E2M1, at, size, st, _stream(stream),
                    ctypes.byref(o))
        elif k_new is None:
            what, code = "gqa_attend_paged", lib.gqa_attend_paged(
                q.data_ptr(), _DTYPES[q.dtype], k.data_ptr(), v.data_ptr(), table.data_ptr(), lengths.data_ptr(),
                out.data_ptr(), B, Hq, Hkv, D, n0, n2, table.shape[1], E2M1, at, size, st, _stream(stream),
                ctypes.byref(o))
        else:
            what, code = "gqa_decode_step_paged", lib.gqa_decode_step_paged_ex(
                q.data_ptr(), k_new.data_ptr(), v_new.data_ptr(), k.data_ptr(), v.data_ptr(), table.data_ptr(),
                lengths.data_ptr(), out.data_ptr(), B, Hq, Hkv, D, n0, n2, table.shape[1], E2M1, at, size, st,
                _stream(stream), ctypes.byref(o))
    _check(code, what)
    return out


def _common_checks(q, k_new, v_new, caches, lengths, out, q_any_dtype=False):
    """Checks shared by the entry points; returns (cache gqa_dtype, out). The
    query and the new keys / values share the cache dtype, except over an E4M3
    cache (bfloat16 then; the attend's query is free)."""
    dev = q.get_device()
    if dev < 0:
        raise ValueError("tensors must be on a CUDA device")
    qt = q.dtype
    if qt not in _DTYPES:
        raise TypeError("q must be float32 or bfloat16")
    code = _cache_code(caches[0][1])
    if code == E4M3:
        if not q_any_dtype and qt != torch.bfloat16:
            raise TypeError("over an E4M3 cache q, k_new and v_new are bfloat16")
        new_dt = torch.bfloat16
    else:
        dt = caches[0][1].dtype if q_any_dtype else qt
        if dt not in _DTYPES:
            raise TypeError("the cache must be float32 or bfloat16")
        new_dt = dt
    news = () if k_new is None else (("k_new", k_new), ("v_new", v_new))
    for name, t in news:
        if t.dtype != new_dt:
            raise TypeError(f"{name} must have dtype {new_dt}")
    for name, t in caches:
        if t.dtype != caches[0][1].dtype:
            raise TypeError(f"{name} must have dtype {caches[0][1].dtype}")
    for name, t in (*news, *caches):
        if t.get_device() != dev:
            raise ValueError(f"{name} is on {t.device}, q on {q.device}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if not q.is_contiguous():
        raise ValueError("q must be contiguous")
    if lengths.dtype != torch.int32 or not lengths.is_contiguous() or lengths.get_device() != dev:
        raise TypeError("lengths must be a contiguous int32 tensor on q's device")
    shape = q.shape
    if out is None:
        out = torch.empty_like(q, dtype=torch.float32)
    elif out.shape != shape or out.dtype != torch.float32 or not out.is_contiguous() or out.get_device() != dev:
        raise ValueError("out must be a contiguous float32 (B, Hq, D) tensor on q's device")
    return code, out


def decode_step(q, k_new, v_new, k_cache, v_cache, lengths, slot_ids=None, *, out=None,
                status=None, kernel="auto", grid_ctas=0, workspace=None, stream=None, sched_pad=None,
                sink=None, window=0, kept_prefix=0, k_scale=None, v_scale=None,
                wait_limit_cycles=0, test_stall=False, k_group_scale=None,
                v_group_scale=None):
    """One decode step on a dense (R, Hkv, Smax, D) cache (continuous batch
    when ``slot_ids`` is given). Appends in place; returns ``out``. A
    ``workspace`` passed in must be zero-filled before its first use (the
    library leaves it zero-filled after every call). ``sink``, ``window`` and
    ``kept_prefix`` are the softmax modifiers of the C header's gqa_options."""
    if k_group_scale is not None or v_group_scale is not None:   # a 4-bit cache
        return _step_e2m1(q, k_new, v_new, k_cache, v_cache, lengths, slot_ids, None, k_scale, v_scale, k_group_scale,
                          v_group_scale, out, status, kernel, grid_ctas, workspace, stream, sched_pad, sink, window,
                          kept_prefix)
    dt, out = _common_checks(q, k_new, v_new, (("k_cache", k_cache), ("v_cache", v_cache)),
                             lengths, out)
    B, Hq, D = q.shape
    R, Hkv, Smax, D2 = k_cache.shape
    if D2 != D or v_cache.shape != k_cache.shape or k_new.shape != (B, Hkv, D) \
            or v_new.shape != (B, Hkv, D):
        raise ValueError("shape mismatch between q, k_new, v_new and the caches")
    if slot_ids is not None and (slot_ids.dtype != torch.int32 or slot_ids.shape != (B,)):
        raise TypeError("slot_ids must be int32 of shape (B,)")
    o = _opts(kernel, grid_ctas, sched_pad, sink, window, kept_prefix, q.device, B, Hq, k_scale, v_scale, Hkv,
              wait_limit_cycles, test_stall)
    lib = _lib.load()
    with _on(q.device):
        need = _need(lib, B, Hq, Hkv, D, dt, kernel, grid_ctas, o, q.device)
        ws = _workspace(q.device, need, stream) if workspace is None else workspace
        code = lib.gqa_decode_step_ex(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
                                      _ptr(lengths), _ptr(slot_ids), _ptr(out), B, Hq, Hkv, D, R, Smax,
                                      dt, _ptr(ws), ws.numel() * ws.element_size(),
                                      _ptr(status), _stream(stream), ctypes.byref(o))
    _check(code, "gqa_decode_step")
    return out


def decode_step_paged(q, k_new, v_new, k_blocks, v_blocks, block_table, lengths, *, out=None,
                      status=None, kernel="auto", grid_ctas=0, workspace=None, stream=None,
                      sched_pad=None, sink=None, window=0, kept_prefix=0, k_scale=None, v_scale=None,
                      wait_limit_cycles=0, test_stall=False, k_group_scale=None,
                      v_group_scale=None):
    """One decode step on a paged cache (num_blocks, Hkv, block_size, D) with
    a (B, max_blocks) int32 block table (-1 = unused). Appends in place."""
    if k_group_scale is not None or v_group_scale is not None:   # a 4-bit cache
        return _step_e2m1(q, k_new, v_new, k_blocks, v_blocks, lengths, None, block_table, k_scale, v_scale, k_group_scale,
                          v_group_scale, out, status, kernel, grid_ctas, workspace, stream, sched_pad, sink, window,
                          kept_prefix)
    dt, out = _common_checks(q, k_new, v_new, (("k_blocks", k_blocks), ("v_blocks", v_blocks)),
                             lengths, out)
    B, Hq, D = q.shape
    NB, Hkv, BS, D2 = k_blocks.shape
    if D2 != D or v_blocks.shape != k_blocks.shape or k_new.shape != (B, Hkv, D) \
            or v_new.shape != (B, Hkv, D):
        raise ValueError("shape mismatch between q, k_new, v_new and the blocks")
    if block_table.dtype != torch.int32 or block_table.dim() != 2 or block_table.shape[0] != B \
            or not block_table.is_contiguous():
        raise TypeError("block_table must be a contiguous int32 (B, max_blocks) tensor")
    MB = block_table.shape[1]
    o = _opts(kernel, grid_ctas, sched_pad, sink, window, kept_prefix, q.device, B, Hq, k_scale, v_scale, Hkv,
              wait_limit_cycles, test_stall)
    lib = _lib.load()
    with _on(q.device):
        need = _need(lib, B, Hq, Hkv, D, dt, kernel, grid_ctas, o, q.device)
        ws = _workspace(q.device, need, stream) if workspace is None else workspace
        code = lib.gqa_decode_step_paged_ex(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_blocks),
                                            _ptr(v_blocks), _ptr(block_table), _ptr(lengths), _ptr(out),
                                            B, Hq, Hkv, D, NB, BS, MB, dt, _ptr(ws),
                                            ws.numel() * ws.element_size(), _ptr(status),
                                            _stream(stream), ctypes.byref(o))
    _check(code, "gqa_decode_step_paged")
    return out


def attend(q, k_cache, v_cache, lengths, slot_ids=None, *, out=None, status=None, kernel="auto",
           grid_ctas=0, workspace=None, stream=None, sched_pad=None, sink=None, window=0,
           kept_prefix=0, k_scale=None, v_scale=None, wait_limit_cycles=0, test_stall=False, k_group_scale=None,
           v_group_scale=None):
    """Read-only attend on a dense (R, Hkv, Smax, D) cache: slots
    ``0..lengths[b]-1`` (1 <= lengths[b] <= Smax), nothing written but ``out``.
    ``q`` (B, Hq, D) is float32 or bfloat16 whatever the cache dtype."""
    if k_group_scale is not None or v_group_scale is not None:   # a 4-bit cache
        return _step_e2m1(q, None, None, k_cache, v_cache, lengths, slot_ids, None, k_scale, v_scale, k_group_scale,
                          v_group_scale, out, status, kernel, grid_ctas, workspace, stream, sched_pad, sink, window,
                          kept_prefix)
    dt, out = _common_checks(q, None, None, (("k_cache", k_cache), ("v_cache", v_cache)),
                             lengths, out, q_any_dtype=True)
    B, Hq, D = q.shape
    R, Hkv, Smax, D2 = k_cache.shape
    if D2 != D or v_cache.shape != k_cache.shape or Hq % Hkv:
        raise ValueError("shape mismatch between q and the caches")
    if slot_ids is not None and (slot_ids.dtype != torch.int32 or slot_ids.shape != (B,)):
        raise TypeError("slot_ids must be int32 of shape (B,)")
    o = _opts(kernel, grid_ctas, sched_pad, sink, window, kept_prefix, q.device, B, Hq, k_scale, v_scale, Hkv,
              wait_limit_cycles, test_stall)
    lib = _lib.load()
    with _on(q.device):
        need = _need(lib, B, Hq, Hkv, D, dt, kernel, grid_ctas, o, q.device)
        ws = _workspace(q.device, need, stream) if workspace is None else workspace
        code = lib.gqa_attend(_ptr(q), _DTYPES[q.dtype], _ptr(k_cache), _ptr(v_cache), _ptr(lengths),
                              _ptr(slot_ids), _ptr(out), B, Hq, Hkv, D, R, Smax, dt, _ptr(ws),
                              ws.numel() * ws.element_size(), _ptr(status), _stream(stream),
                              ctypes.byref(o))
    _check(code, "gqa_attend")
    return out


def attend_paged(q, k_blocks, v_blocks, block_table, lengths, *, out=None, status=None,
                 kernel="auto", grid_ctas=0, workspace=None, stream=None, sched_pad=None,
                 sink=None, window=0, kept_prefix=0, k_scale=None, v_scale=None,
                wait_limit_cycles=0, test_stall=False, k_group_scale=None,
                 v_group_scale=None):
    """Read-only attend on a paged cache (num_blocks, Hkv, block_size, D)."""
    if k_group_scale is not None or v_group_scale is not None:   # a 4-bit cache
        return _step_e2m1(q, None, None, k_blocks, v_blocks, lengths, None, block_table, k_scale, v_scale, k_group_scale,
                          v_group_scale, out, status, kernel, grid_ctas, workspace, stream, sched_pad, sink, window,
                          kept_prefix)
    dt, out = _common_checks(q, None, None, (("k_blocks", k_blocks), ("v_blocks", v_blocks)),
                             lengths, out, q_any_dtype=True)
    B, Hq, D = q.shape
    NB, Hkv, BS, D2 = k_blocks.shape
    if D2 != D or v_blocks.shape != k_blocks.shape or Hq % Hkv:
        raise ValueError("shape mismatch between q and the blocks")
    if block_table.dtype != torch.int32 or block_table.dim() != 2 or block_table.shape[0] != B \
            or not block_table.is_contiguous():
        raise TypeError("block_table must be a contiguous int32 (B, max_blocks) tensor")
    o = _opts(kernel, grid_ctas, sched_pad, sink, window, kept_prefix, q.device, B, Hq, k_scale, v_scale, Hkv,
              wait_limit_cycles, test_stall)
    lib = _lib.load()
    with _on(q.device):
        need = _need(lib, B, Hq, Hkv, D, dt, kernel, grid_ctas, o, q.device)
        ws = _workspace(q.device, need, stream) if workspace is None else workspace
        code = lib.gqa_attend_paged(_ptr(q), _DTYPES[q.dtype], _ptr(k_blocks), _ptr(v_blocks),
                                    _ptr(block_table), _ptr(lengths), _ptr(out), B, Hq, Hkv, D, NB, BS,
                                    block_table.shape[1], dt, _ptr(ws),
                                    ws.numel() * ws.element_size(), _ptr(status), _stream(stream),
                                    ctypes.byref(o))
    _check(code, "gqa_attend_paged")
    return out


def _multi_checks(q, k_new, v_new, caches, lengths, cu_q, out):
    dt, out = _common_checks(q, k_new, v_new, caches, lengths, out)
    if cu_q.dtype != torch.int32 or cu_q.dim() != 1 or cu_q.shape[0] != lengths.shape[0] + 1 \
            or not cu_q.is_contiguous() or cu_q.device != q.device:
        raise TypeError("cu_q must be a contiguous int32 (B + 1,) tensor on q's device")
    return dt, out


def decode_multi(q, k_new, v_new, k_cache, v_cache, lengths, cu_q, slot_ids=None, *, max_q_len,
                 out=None, status=None, kernel="auto", grid_ctas=0, workspace=None, stream=None,
                 sched_pad=None, sink=None, window=0, kept_prefix=0, k_scale=None,
                 v_scale=None, wait_limit_cycles=0, test_stall=False):
    """Multi-token step on a dense (R, Hkv, Smax, D) cache: the packed tokens
    cu_q[b] .. cu_q[b+1]-1 of row b (q (T, Hq, D), k_new / v_new (T, Hkv, D))
    are appended at slots lengths[b] + i and token i attends slots
    0 .. lengths[b] + i. ``max_q_len`` bounds every q_len. Over an E4M3
    cache q, k_new and v_new are bfloat16 and ``k_scale`` / ``v_scale`` are
    required, as in :func:`decode_step`. Returns out (T, Hq, D)."""
    dt, out = _multi_checks(q, k_new, v_new, (("k_cache", k_cache), ("v_cache", v_cache)), lengths,
                            cu_q, out)
    T, Hq, D = q.shape
    B = lengths.shape[0]
    R, Hkv, Smax, D2 = k_cache.shape
    if D2 != D or v_cache.shape != k_cache.shape or k_new.shape != (T, Hkv, D) or v_new.shape != (T, Hkv, D):
        raise ValueError("shape mismatch between q, k_new, v_new and the caches")
    if slot_ids is not None and (slot_ids.dtype != torch.int32 or slot_ids.shape != (B,)):
        raise TypeError("slot_ids must be int32 of shape (B,)")
    o = _opts(kernel, grid_ctas, sched_pad, sink, window, kept_prefix, q.device, B, Hq, k_scale, v_scale, Hkv,
              wait_limit_cycles, test_stall)
    lib = _lib.load()
    with _on(q.device):
        need = lib.gqa_workspace_bytes_multi(B, Hq, Hkv, D, dt, int(max_q_len), ctypes.byref(o))
        ws = _workspace(q.device, need, stream) if workspace is None else workspace
        code = lib.gqa_decode_multi(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
                                    _ptr(lengths), _ptr(cu_q), _ptr(slot_ids), _ptr(out), B, T, int(max_q_len),
                                    Hq, Hkv, D, R, Smax, dt, _ptr(ws), ws.numel() * ws.element_size(),
                                    _ptr(status), _stream(stream), ctypes.byref(o))
    _check(code, "gqa_decode_multi")
    return out


def decode_multi_paged(q, k_new, v_new, k_blocks, v_blocks, block_table, lengths, cu_q, *, max_q_len,
                       out=None, status=None, kernel="auto", grid_ctas=0, workspace=None, stream=None,
                       sched_pad=None, sink=None, window=0, kept_prefix=0, k_scale=None,
                       v_scale=None, wait_limit_cycles=0, test_stall=False):
    """Multi-token step on a paged cache (num_blocks, Hkv, block_size, D)."""
    dt, out = _multi_checks(q, k_new, v_new, (("k_blocks", k_blocks), ("v_blocks", v_blocks)), lengths,
                            cu_q, out)
    T, Hq, D = q.shape
    B = lengths.shape[0]
    NB, Hkv, BS, D2 = k_blocks.shape
    if D2 != D or v_blocks.shape != k_blocks.shape or k_new.shape != (T, Hkv, D) or v_new.shape != (T, Hkv, D):
        raise ValueError("shape mismatch between q, k_new, v_new and the blocks")
    if block_table.dtype != torch.int32 or block_table.dim() != 2 or block_table.shape[0] != B \
            or not block_table.is_contiguous():
        raise TypeError("block_table must be a contiguous int32 (B, max_blocks) tensor")
    o = _opts(kernel, grid_ctas, sched_pad, sink, window, kept_prefix, q.device, B, Hq, k_scale, v_scale, Hkv,
              wait_limit_cycles, test_stall)
    lib = _lib.load()
    with _on(q.device):
        need = lib.gqa_workspace_bytes_multi(B, Hq, Hkv, D, dt, int(max_q_len), ctypes.byref(o))
        ws = _workspace(q.device, need, stream) if workspace is None else workspace
        code = lib.gqa_decode_multi_paged(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_blocks), _ptr(v_blocks),
                                          _ptr(block_table), _ptr(lengths), _ptr(cu_q), _ptr(out), B, T,
                                          int(max_q_len), Hq, Hkv, D, NB, BS, block_table.shape[1], dt,
                                          _ptr(ws), ws.numel() * ws.element_size(), _ptr(status),
                                          _stream(stream), ctypes.byref(o))
    _check(code, "gqa_decode_multi_paged")
    return out


# ---- writing and reading a cache, block selection ----

def _int32(name, t, n, dev):
    if t.dtype != torch.int32 or t.shape != (n,) or not t.is_contiguous() or t.get_device() != dev:
        raise TypeError(f"{name} must be a contiguous int32 ({n},) tensor on the other tensors' device")


def _rows_checks(caches, lengths, cu_q, slot_ids, block_table, groups, D):
    """Checks shared by append and read; returns the cache's gqa_dtype."""
    (_, k), (_, v) = caches
    dev = k.get_device()
    if dev < 0:
        raise ValueError("tensors must be on a CUDA device")
    shape = k.shape
    if v.shape != shape or v.dtype != k.dtype or v.get_device() != dev or len(shape) != 4:
        raise ValueError("the two caches must be 4-dimensional and alike")
    if not (k.is_contiguous() and v.is_contiguous()):
        raise ValueError("the caches must be contiguous")
    if groups[0] is not None or groups[1] is not None:
        _group_scales(caches, *groups, D)
        code = E2M1
    else:
        code = _cache_code(k)
        if shape[3] != D:
            raise ValueError("shape mismatch between the vectors and the caches")
    B = lengths.shape[0]
    _int32("lengths", lengths, B, dev)
    _int32("cu_q", cu_q, B + 1, dev)
    if slot_ids is not None:
        _int32("slot_ids", slot_ids, B, dev)
    if block_table is not None and (block_table.dtype != torch.int32 or block_table.dim() != 2
                                    or block_table.shape[0] != B or not block_table.is_contiguous()
                                    or block_table.get_device() != dev):
        raise TypeError("block_table must be a contiguous int32 (B, max_blocks) tensor on the caches' device")
    return code


def _rows_opts(code, Hkv, device, k_scale, v_scale, groups):
    """The options that carry a quantised cache's scales (None for the others)."""
    if code < E4M3:
        return None
    return ctypes.byref(_opts("auto", 0, device=device, k_scale=k_scale, v_scale=v_scale, Hkv=Hkv,
                              k_group_scale=groups[0], v_group_scale=groups[1]))


def _status_checks(status, device):
    if status is not None and (status.dtype != torch.int32 or status.device != device):
        raise TypeError("status must be an int32 tensor on the caches' device")


def _append(k_new, v_new, k, v, block_table, lengths, cu_q, slot_ids, scales, groups, k_bounds, status, stream,
            names):
    if k_new.dim() != 3 or v_new.shape != k_new.shape:
        raise ValueError("k_new and v_new must both be (T, Hkv, D)")
    T, Hkv, D = k_new.shape
    code = _rows_checks(((names[0], k), (names[1], v)), lengths, cu_q, slot_ids, block_table, groups, D)
    dev = k.get_device()
    if k_new.dtype not in _DTYPES or v_new.dtype != k_new.dtype:
        raise TypeError("k_new and v_new must both be float32 or bfloat16")
    for t in (k_new, v_new):
        if t.get_device() != dev or not t.is_contiguous():
            raise ValueError("k_new and v_new must be contiguous and on the caches' device")
    n0, heads, n2, _ = k.shape
    if heads != Hkv:
        raise ValueError("shape mismatch between k_new and the caches")
    device = k.device
    if status is not None:
        _status_checks(status, device)
    block = 0
    if k_bounds is not None:
        if block_table is not None:
            shape = (n0, Hkv, 2, D)
        else:
            if k_bounds.dim() != 5 or k_bounds.shape[2] < 1 or n2 % k_bounds.shape[2]:
                raise ValueError("k_bounds must be (R, Hkv, NB, 2, D) with NB a divisor of Smax")
            block = n2 // k_bounds.shape[2]
            shape = (n0, Hkv, k_bounds.shape[2], 2, D)
        if k_bounds.dtype != torch.bfloat16 or k_bounds.shape != shape or not k_bounds.is_contiguous() \
                or k_bounds.get_device() != dev:
            raise TypeError(f"k_bounds must be a contiguous bfloat16 {shape} tensor on the caches' device")
    o = _rows_opts(code, Hkv, device, *scales, groups)
    lib = _lib.load()
    B = lengths.shape[0]
    with _on(device):
        if block_table is not None:
            what = "gqa_append_paged"
            rc = lib.gqa_append_paged(_ptr(k_new), _ptr(v_new), _DTYPES[k_new.dtype], _ptr(k), _ptr(v),
                                      _ptr(block_table), _ptr(lengths), _ptr(cu_q), _ptr(k_bounds), B, T, Hkv, D, n0,
                                      n2, block_table.shape[1], code, _ptr(status), _stream(stream, device), o)
        else:
            what = "gqa_append"
            rc = lib.gqa_append(_ptr(k_new), _ptr(v_new), _DTYPES[k_new.dtype], _ptr(k), _ptr(v), _ptr(lengths),
                                _ptr(cu_q), _ptr(slot_ids), _ptr(k_bounds), block, B, T, Hkv, D, n0, n2, code,
                                _ptr(status), _stream(stream, device), o)
    _check(rc, what)


def append(k_new, v_new, k_cache, v_cache, lengths, cu_q, slot_ids=None, *, k_bounds=None, k_scale=None,
           v_scale=None, k_group_scale=None, v_group_scale=None, status=None, stream=None):
    """Writes the packed tokens cu_q[b] .. cu_q[b+1]-1 (``k_new``, ``v_new``
    (T, Hkv, D), float32 or bfloat16) into slots lengths[b] .. of row b of a
    dense (R, Hkv, Smax, D) cache, in place, rounded to its type. Tokens behind
    the last row are ignored. ``k_bounds``, a bfloat16 (R, Hkv, NB, 2, D)
    tensor, follows the smallest and largest key of every block of Smax // NB
    slots for :func:`select_blocks`."""
    _append(k_new, v_new, k_cache, v_cache, None, lengths, cu_q, slot_ids, (k_scale, v_scale),
            (k_group_scale, v_group_scale), k_bounds, status, stream, ("k_cache", "v_cache"))


def append_paged(k_new, v_new, k_blocks, v_blocks, block_table, lengths, cu_q, *, k_bounds=None, k_scale=None,
                 v_scale=None, k_group_scale=None, v_group_scale=None, status=None, stream=None):
    """:func:`append` into a paged cache (num_blocks, Hkv, block_size, D);
    ``k_bounds`` is (num_blocks, Hkv, 2, D)."""
    _append(k_new, v_new, k_blocks, v_blocks, block_table, lengths, cu_q, None, (k_scale, v_scale),
            (k_group_scale, v_group_scale), k_bounds, status, stream, ("k_blocks", "v_blocks"))


def _read(k, v, block_table, lengths, cu_q, T, slot_ids, dtype, k_out, v_out, scales, groups, status, stream, names):
    if dtype not in _DTYPES:
        raise TypeError("dtype must be torch.float32 or torch.bfloat16")
    D = k.shape[-1] * (2 if groups[0] is not None or groups[1] is not None else 1)
    code = _rows_checks(((names[0], k), (names[1], v)), lengths, cu_q, slot_ids, block_table, groups, D)
    device, dev = k.device, k.get_device()
    if status is not None:
        _status_checks(status, device)
    n0, Hkv, n2, _ = k.shape
    T, shape = int(T), (int(T), Hkv, D)
    for name, t in (("k_out", k_out), ("v_out", v_out)):
        if t is not None and (t.shape != shape or t.dtype != dtype or t.get_device() != dev or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous {dtype} {shape} tensor on the caches' device")
    if k_out is None or v_out is None:
        with torch.cuda.stream(stream) if stream is not None else _HERE:
            k_out = torch.empty(shape, dtype=dtype, device=device) if k_out is None else k_out
            v_out = torch.empty(shape, dtype=dtype, device=device) if v_out is None else v_out
    o = _rows_opts(code, Hkv, device, *scales, groups)
    lib = _lib.load()
    B = lengths.shape[0]
    with _on(device):
        if block_table is not None:
            what = "gqa_read_paged"
            rc = lib.gqa_read_paged(_ptr(k), _ptr(v), _ptr(block_table), _ptr(lengths), _ptr(cu_q), _ptr(k_out),
                                    _ptr(v_out), _DTYPES[dtype], B, T, Hkv, D, n0, n2, block_table.shape[1], code,
                                    _ptr(status), _stream(stream, device), o)
        else:
            what = "gqa_read"
            rc = lib.gqa_read(_ptr(k), _ptr(v), _ptr(lengths), _ptr(cu_q), _ptr(slot_ids), _ptr(k_out), _ptr(v_out),
                              _DTYPES[dtype], B, T, Hkv, D, n0, n2, code, _ptr(status), _stream(stream, device), o)
    _check(rc, what)
    return k_out, v_out


def read(k_cache, v_cache, lengths, cu_q, T, slot_ids=None, *, dtype=torch.bfloat16, k_out=None, v_out=None,
         k_scale=None, v_scale=None, k_group_scale=None, v_group_scale=None, status=None, stream=None):
    """Slots lengths[b] .. lengths[b] + cu_q[b+1] - cu_q[b] - 1 of row b of a
    dense cache as vectors: two (T, Hkv, D) tensors of ``dtype``, packed by
    ``cu_q`` (what :func:`append` with the same arguments wrote, rounded to the
    cache's type). Packed rows of no batch row are left as they were."""
    return _read(k_cache, v_cache, None, lengths, cu_q, T, slot_ids, dtype, k_out, v_out, (k_scale, v_scale),
                 (k_group_scale, v_group_scale), status, stream, ("k_cache", "v_cache"))


def read_paged(k_blocks, v_blocks, block_table, lengths, cu_q, T, *, dtype=torch.bfloat16, k_out=None, v_out=None,
               k_scale=None, v_scale=None, k_group_scale=None, v_group_scale=None, status=None, stream=None):
    """:func:`read` from a paged cache (num_blocks, Hkv, block_size, D)."""
    return _read(k_blocks, v_blocks, block_table, lengths, cu_q, T, None, dtype, k_out, v_out, (k_scale, v_scale),
                 (k_group_scale, v_group_scale), status, stream, ("k_blocks", "v_blocks"))


class Selection:
    """The blocks that :func:`select_blocks` kept: ``ids`` (B, Hkv, n_select)
    int32, ascending, then -1; ``table`` (B * Hkv, n_select), the same blocks in
    the cache seen as a pool of one-head blocks; ``lengths`` (B * Hkv,), the
    slots they hold."""

    def __init__(self, B, Hkv, n_select, block_size, device):
        self.B, self.Hkv, self.n_select, self.block_size = B, Hkv, n_select, block_size
        self._n = B * Hkv * n_select
        self._pool = None   # (rows, blocks a row; paged: blocks, 0) of the cache it was made over; None: not made yet
        self._buf = torch.empty(2 * self._n + B * Hkv, dtype=torch.int32, device=device)

    @property
    def ids(self):
        return self._buf[:self._n].view(self.B, self.Hkv, self.n_select)

    @property
    def table(self):
        return self._buf[self._n:2 * self._n].view(self.B * self.Hkv, self.n_select)

    @property
    def lengths(self):
        return self._buf[2 * self._n:]

    def _ptrs(self):
        at = self._buf.data_ptr()
        return at, at + 4 * self._n, at + 8 * self._n


def _select(q, k_bounds, block_table, lengths, n_select, slot_ids, block_size, n_first, n_last, selection, status,
            stream):
    dev = q.get_device()
    if dev < 0:
        raise ValueError("tensors must be on a CUDA device")
    if q.dtype not in _DTYPES or q.dim() != 3:
        raise TypeError("q must be a float32 or bfloat16 (B, Hq, D) tensor")
    B, Hq, D = q.shape
    kb = k_bounds.shape
    if k_bounds.dtype != torch.bfloat16 or len(kb) != (5 if block_table is None else 4) or kb[-2] != 2 or kb[-1] != D:
        raise TypeError("k_bounds must be bfloat16, (R, Hkv, NB, 2, D) for a dense cache and (num_blocks, Hkv, 2, D) "
                        "for a paged one")
    Hkv = kb[1]
    if Hq % Hkv:
        raise ValueError("Hq must be a multiple of Hkv")
    _plain(dev, q, k_bounds)
    _int32("lengths", lengths, B, dev)
    if slot_ids is not None:
        _int32("slot_ids", slot_ids, B, dev)
    if block_table is not None and (block_table.dtype != torch.int32 or block_table.dim() != 2
                                    or block_table.shape[0] != B or not block_table.is_contiguous()
                                    or block_table.get_device() != dev):
        raise TypeError("block_table must be a contiguous int32 (B, max_blocks) tensor on q's device")
    device = q.device
    if status is not None:
        _status_checks(status, device)
    n_select = int(n_select)
    if selection is None:
        if n_select < 1 or block_size < 1:
            raise ValueError("n_select and block_size must be positive")
        with torch.cuda.stream(stream) if stream is not None else _HERE:
            selection = Selection(B, Hkv, n_select, int(block_size), device)
    elif (selection.B, selection.Hkv, selection.n_select, selection.block_size) != (B, Hkv, n_select, int(block_size)) \
            or selection._buf.device != device:
        raise ValueError("selection was made for other sizes")
    ids, table, slots = selection._ptrs()
    selection._pool = None
    lib = _lib.load()
    with _on(device):
        if block_table is None:
            what = "gqa_select_blocks"
            rc = lib.gqa_select_blocks(_ptr(q), _DTYPES[q.dtype], _ptr(k_bounds), _ptr(lengths), _ptr(slot_ids), ids,
                                       table, slots, B, Hq, Hkv, D, kb[0], kb[2],
                                       selection.block_size, n_select, int(n_first), int(n_last), _ptr(status),
                                       _stream(stream, device))
        else:
            what = "gqa_select_blocks_paged"
            rc = lib.gqa_select_blocks_paged(_ptr(q), _DTYPES[q.dtype], _ptr(k_bounds), _ptr(block_table),
                                             _ptr(lengths), ids, table, slots, B, Hq, Hkv, D, kb[0],
                                             selection.block_size, block_table.shape[1], n_select, int(n_first),
                                             int(n_last), _ptr(status), _stream(stream, device))
    _check(rc, what)
    selection._pool = (kb[0], kb[2] if block_table is None else 0)
    return selection


def select_blocks(q, k_bounds, lengths, n_select, slot_ids=None, *, block_size, n_first=1, n_last=1, selection=None,
                  status=None, stream=None):
    """Chooses, for every (row, cache head) of a dense cache, at most
    ``n_select`` blocks of ``block_size`` slots: the first ``n_first`` and the
    last ``n_last`` of the row's ceil(lengths[b] / block_size) blocks, and those
    whose key bounds (``k_bounds`` (R, Hkv, NB, 2, D), see :func:`append`) allow
    the largest score summed over the cache head's queries. ``lengths`` counts
    the valid slots, as in :func:`attend`. Returns a :class:`Selection`
    (``selection``, one of the same sizes, is filled instead when given)."""
    return _select(q, k_bounds, None, lengths, n_select, slot_ids, block_size, n_first, n_last, selection, status,
                   stream)


def select_blocks_paged(q, k_bounds, block_table, lengths, n_select, *, block_size, n_first=1, n_last=1,
                        selection=None, status=None, stream=None):
    """:func:`select_blocks` over a paged cache: a block is a page of
    ``block_size`` slots, ``k_bounds`` is (num_blocks, Hkv, 2, D)."""
    return _select(q, k_bounds, block_table, lengths, n_select, None, block_size, n_first, n_last, selection, status,
                   stream)


def attend_selected(q, k_cache, v_cache, selection, *, out=None, status=None, kernel="auto", grid_ctas=0,
                    workspace=None, stream=None, sched_pad=None, k_scale=None, v_scale=None, k_group_scale=None,
                    v_group_scale=None):
    """Read-only attend over the kept blocks of a dense (R, Hkv, Smax, D) or
    paged (num_blocks, Hkv, block_size, D) float32, bfloat16 or E2M1 cache:
    every query head attends the slots of its cache head's blocks in
    ``selection``, and nothing is written but ``out`` (B, Hq, D) float32."""
    if stream is not None and out is None:
        with torch.cuda.stream(stream):
            out = torch.empty(q.shape, dtype=torch.float32, device=q.device)
    sel = selection
    if k_group_scale is not None or v_group_scale is not None:
        dt = E2M1
        _plain(_check_e2m1(q, k_cache, v_cache, k_group_scale, v_group_scale, out), sel._buf)
    else:
        dt, out = _common_checks(q, None, None, (("k_cache", k_cache), ("v_cache", v_cache)), sel._buf, out,
                                 q_any_dtype=True)
    B, Hq, D = q.shape
    n0, Hkv, n2, D2 = k_cache.shape
    if (D2 * 2 if dt == E2M1 else D2) != D or v_cache.shape != k_cache.shape or (B, Hkv) != (sel.B, sel.Hkv) \
            or Hq % Hkv or sel._pool is None \
            or (n0, n2) != (sel._pool[0], (sel._pool[1] or 1) * sel.block_size):
        raise ValueError("shape mismatch between q, the caches and the selection")
    device = q.device
    if status is not None:
        _status_checks(status, device)
    if workspace is not None:
        _plain(device.index, workspace)
    o = _opts(kernel, grid_ctas, sched_pad, device=device, k_scale=k_scale, v_scale=v_scale, Hkv=Hkv,
              k_group_scale=k_group_scale, v_group_scale=v_group_scale)
    lib = _lib.load()
    _, table, slots = sel._ptrs()
    with _on(device):
        need = _need(lib, B * Hkv, Hq // Hkv, 1, D, dt, kernel, grid_ctas, o, device)
        ws = _workspace(device, need, stream) if workspace is None else workspace
        if out is None:
            out = torch.empty_like(q, dtype=torch.float32)
        rc = lib.gqa_attend_selected(_ptr(q), _DTYPES[q.dtype], _ptr(k_cache), _ptr(v_cache), table, slots, _ptr(out),
                                     B, Hq, Hkv, D, n0 * Hkv * (n2 // sel.block_size), sel.block_size, sel.n_select,
                                     dt, _ptr(ws), ws.numel() * ws.element_size(), _ptr(status),
                                     _stream(stream, device), ctypes.byref(o))
    _check(rc, "gqa_attend_selected")
    return out


def validate_multi(lengths, cu_q, T, *, slot_ids=None, R=None, Smax=None, block_table=None,
                   num_blocks=None, block_size=None, stream=None) -> bool:
    """Full content check on the GPU for a multi-token step (synchronous)."""
    B = lengths.shape[0]
    res = torch.empty(1, dtype=torch.int32, device=lengths.device)
    lib = _lib.load()
    if block_table is not None:
        code = lib.gqa_validate_multi(_ptr(lengths), _ptr(cu_q), None, _ptr(block_table), B, T, 0, 0,
                                      num_blocks, block_size, block_table.shape[1], _ptr(res), _stream(stream))
    else:
        code = lib.gqa_validate_multi(_ptr(lengths), _ptr(cu_q), _ptr(slot_ids), None, B, T, R, Smax, 0, 0, 0,
                                      _ptr(res), _stream(stream))
    if code == INVALID_ARGUMENT:
        return False
    _check(code, "gqa_validate_multi")
    return True


def _validate(fn, what, lengths, slot_ids, R, Smax, block_table, num_blocks, block_size, stream):
    B = lengths.shape[0]
    res = torch.empty(1, dtype=torch.int32, device=lengths.device)
    if block_table is not None:
        code = fn(_ptr(lengths), None, _ptr(block_table), B, 0, 0, num_blocks, block_size,
                  block_table.shape[1], _ptr(res), _stream(stream))
    else:
        code = fn(_ptr(lengths), _ptr(slot_ids), None, B, R, Smax, 0, 0, 0, _ptr(res),
                  _stream(stream))
    if code == INVALID_ARGUMENT:
        return False
    _check(code, what)
    return True


def validate(lengths, *, slot_ids=None, R=None, Smax=None, block_table=None, num_blocks=None,
             block_size=None, stream=None) -> bool:
    """Full content check on the GPU for the decode step (synchronous). True
    when valid."""
    return _validate(_lib.load().gqa_validate, "gqa_validate", lengths, slot_ids, R, Smax,
                     block_table, num_blocks, block_size, stream)


def validate_attend(lengths, *, slot_ids=None, R=None, Smax=None, block_table=None,
                    num_blocks=None, block_size=None, stream=None) -> bool:
    """Full content check on the GPU for the read-only attend (synchronous)."""
    return _validate(_lib.load().gqa_validate_attend, "gqa_validate_attend", lengths, slot_ids, R,
                     Smax, block_table, num_blocks, block_size, stream)


def trace_enable(on: bool = True) -> bool:
    return bool(_lib.load().gqa_trace_enable(int(on)))


def trace_collect() -> dict:
    """{kernel name: (launches, total ms)} since the previous collect."""
    lib = _lib.load()
    n = 4
    launches = (ctypes.c_int64 * n)()
    ms = (ctypes.c_double * n)()
    _check(lib.gqa_trace_collect(n, launches, ms), "gqa_trace_collect")
    return {lib.gqa_kernel_name(k).decode(): (launches[k], ms[k]) for k in range(n)}
