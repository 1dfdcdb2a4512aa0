"""ctypes binding of librlmoe.so (include/rl_moe.h).

Argument marshalling only: every function here has the name of a C entry point, turns
tensors (or None) into raw pointers, calls the library, and raises RlError on a non-OK
status.  All compute happens in the CUDA kernels.  The library must have been built
(`quantized_moe_expert_rl_gb300.build.build()`); loading fails loudly if it is missing.
"""
from __future__ import annotations

import ctypes
import os

from .build import LIB

RL_OK, RL_ERR_INVALID, RL_ERR_UNSUPPORTED, RL_ERR_CUDA, RL_ERR_TIMEOUT = 0, 1, 2, 3, 4
RL_NO_EARLY_OUT = 0x7FFFFFFF
RL_DEVERR_SLOT_ALIGN, RL_DEVERR_WAIT_TIMEOUT, RL_DEVERR_BAD_ID, RL_DEVERR_MISSING, RL_DEVERR_RANGE = 1, 2, 4, 8, 16
RL_DEVERR_NAN = 32
STATUS_NAMES = {0: "RL_OK", 1: "RL_ERR_INVALID", 2: "RL_ERR_UNSUPPORTED", 3: "RL_ERR_CUDA", 4: "RL_ERR_TIMEOUT"}

# every symbol include/rl_moe.h declares
EXPORTS = ("rl_abi_version", "rl_last_error", "rl_record_bytes", "rl_rmsnorm", "rl_route_workspace_bytes",
           "rl_route", "rl_resolve_slots", "moe_decode_workspace_bytes", "moe_decode",
           "rl_build_pairs_workspace_bytes", "rl_build_pairs", "moe_prefill_workspace_bytes",
           "moe_prefill_chunk", "moe_prefill_chunk_f32", "moe_decode_static", "moe_decode_stack_workspace_bytes",
           "moe_decode_stack", "rl_fill_workspace_bytes", "rl_fill_missing", "rl_host_device_pointer",
           "moe_decode_stack_fill", "moe_decode_layer", "moe_decode_tokens_workspace_bytes", "moe_decode_tokens",
           "rl_add_rmsnorm", "rl_q4_matvec", "rl_logprobs_workspace_bytes", "rl_logprobs", "rl_f8_matmul", "rl_f8_gated",
           "rl_sample")

RL_F32, RL_F16, RL_BF16, RL_F8_E4M3 = 0, 1, 2, 3
RL_MAX_DECODE_TOKENS = 32


class RlShape(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("n_experts", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("inter", ctypes.c_int32), ("n_layers", ctypes.c_int32)]

    @classmethod
    def of(cls, hidden, n_experts, top_k, inter, n_layers):
        return cls(hidden, n_experts, top_k, inter, n_layers)


class RlError(RuntimeError):
    def __init__(self, status: int, fn: str, msg: str):
        super().__init__(f"{fn}: {STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


_lib = None


def load(path: str | None = None) -> ctypes.CDLL:
    """Load librlmoe.so (no fallback: raises if the CUDA library was not built)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB
    if not os.path.exists(p):
        raise RuntimeError(f"CUDA library {p} not built; run quantized_moe_expert_rl_gb300.build.build()")
    L = ctypes.CDLL(p)
    i32, u64p, vp, sz, f32 = ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_float
    shp = ctypes.POINTER(RlShape)
    sig = {
        "rl_abi_version": (i32, []),
        "rl_last_error": (ctypes.c_char_p, []),
        "rl_record_bytes": (sz, [shp]),
        "rl_rmsnorm": (i32, [vp, vp, i32, i32, f32, vp]),
        "rl_route_workspace_bytes": (sz, [shp, i32]),
        "rl_route": (i32, [shp, i32, i32, vp, f32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
        "rl_resolve_slots": (i32, [shp, i32, i32, vp, vp, vp, vp]),
        "moe_decode_workspace_bytes": (sz, [shp]),
        "moe_decode": (i32, [shp, i32, vp, f32, vp, vp, vp, vp, i32, vp, vp, sz, vp]),
        "moe_decode_static": (i32, [shp, i32, vp, f32, vp, vp, vp, vp, i32, vp, vp]),
        "moe_decode_stack_workspace_bytes": (sz, [shp]),
        "moe_decode_stack": (i32, [shp, i32, i32, vp, f32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, vp, vp, sz,
                                   vp]),
        "rl_build_pairs_workspace_bytes": (sz, [shp, i32]),
        "rl_build_pairs": (i32, [shp, i32, i32, vp, vp, vp, vp, vp, vp, sz, vp]),
        "moe_prefill_workspace_bytes": (sz, [shp, i32]),
        "moe_prefill_chunk": (i32, [shp, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, i32, vp, vp, sz, vp]),
        "moe_prefill_chunk_f32": (i32, [shp, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, i32, vp, vp, sz, vp]),
        "moe_decode_stack_fill": (i32, [shp, i32, i32, vp, f32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                        vp, vp, sz, vp]),
        "moe_decode_layer": (i32, [shp, i32, vp, f32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
        "moe_decode_tokens_workspace_bytes": (sz, [shp, i32]),
        "moe_decode_tokens": (i32, [shp, i32, i32, vp, f32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, vp, sz,
                                    vp]),
        "rl_add_rmsnorm": (i32, [vp, vp, vp, i32, i32, i32, f32, vp, vp, vp, vp, i32, vp]),
        "rl_q4_matvec": (i32, [vp, vp, i32, i32, i32, vp, i32, vp, i32, vp, i32, i32, vp]),
        "rl_f8_matmul": (i32, [vp, vp, i32, i32, vp, vp, i32, vp, vp, i32, i32, vp, vp]),
        "rl_f8_gated": (i32, [vp, vp, vp, vp, i32, i32, vp, vp, i32, vp, i32, vp, vp, i32, vp, vp]),
        "rl_sample": (i32, [vp, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp]),
        "rl_logprobs_workspace_bytes": (sz, [i32, i32, i32]),
        "rl_logprobs": (i32, [vp, i32, i32, i32, vp, vp, vp, i32, vp, vp, vp, sz, vp]),
        "rl_fill_workspace_bytes": (sz, [shp]),
        "rl_fill_missing": (i32, [shp, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
        "rl_host_device_pointer": (i32, [vp, ctypes.POINTER(ctypes.c_uint64)]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype, fn.argtypes = res, args
    del u64p
    if path is None:
        _lib = L
    return L


def ptr(t) -> int | None:
    """Raw address of a device tensor / int / None (NULL).  The library reads every buffer as
    a dense array on the device, so a strided view or a host tensor is refused here rather
    than read wrongly."""
    if t is None:
        return None
    if isinstance(t, int):
        return t or None
    if not t.is_contiguous():
        raise ValueError(f"tensor of shape {tuple(t.shape)} and strides {t.stride()} is not contiguous")
    if t.device.type != "cuda":
        raise ValueError(f"tensor on {t.device} passed where a device buffer is expected")
    return t.data_ptr() or None


_current = None  # (device index of the calling thread, raw current stream of a device)


def _cuda():
    """torch's raw lookups of the current device and stream: the Stream object that
    torch.cuda.current_stream() builds costs more (4 us) than a whole launch."""
    global _current
    if _current is None:
        import torch
        torch.cuda.init()
        _current = (torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream)
    return _current


def _stream(s) -> int | None:
    if s is None:
        device, raw = _current or _cuda()
        return raw(device()) or None
    if isinstance(s, int):
        return s or None
    return s.cuda_stream or None


def _check(fn: str, st: int) -> None:
    if st != RL_OK:
        raise RlError(st, fn, load().rl_last_error().decode())


def rl_abi_version() -> int:
    return load().rl_abi_version()


def rl_record_bytes(shape: RlShape) -> int:
    return load().rl_record_bytes(ctypes.byref(shape))


def rl_rmsnorm(x, xn, T, H, eps, stream=None):
    _check("rl_rmsnorm", load().rl_rmsnorm(ptr(x), ptr(xn), T, H, eps, _stream(stream)))


def rl_route_workspace_bytes(shape, T) -> int:
    return load().rl_route_workspace_bytes(ctypes.byref(shape), T)


def rl_route(shape, layer, T, x, norm_eps, w_router, bias, residency, ids, weights, slots, miss, ctrl,
             logits_out=None, ws=None, ws_bytes=0, stream=None):
    _check("rl_route", load().rl_route(ctypes.byref(shape), layer, T, ptr(x), float(norm_eps), ptr(w_router), ptr(bias),
                                       ptr(residency), ptr(ids), ptr(weights), ptr(slots), ptr(miss), ptr(ctrl),
                                       ptr(logits_out), ptr(ws), ws_bytes, _stream(stream)))


def rl_fill_workspace_bytes(shape) -> int:
    return load().rl_fill_workspace_bytes(ctypes.byref(shape))


def rl_fill_missing(shape, layer, T, ids, slots, residency, src, dst, filled, first_early_out, ctrl, ws, ws_bytes,
                    stream=None):
    _check("rl_fill_missing", load().rl_fill_missing(ctypes.byref(shape), layer, T, ptr(ids), ptr(slots),
                                                     ptr(residency), ptr(src), ptr(dst), ptr(filled),
                                                     ptr(first_early_out), ptr(ctrl), ptr(ws), ws_bytes,
                                                     _stream(stream)))


def rl_host_device_pointer(host_ptr: int) -> int:
    out = ctypes.c_uint64(0)
    _check("rl_host_device_pointer", load().rl_host_device_pointer(host_ptr, ctypes.byref(out)))
    return int(out.value)


def rl_resolve_slots(shape, layer, T, ids, residency, slots, stream=None):
    _check("rl_resolve_slots", load().rl_resolve_slots(ctypes.byref(shape), layer, T, ptr(ids), ptr(residency),
                                                       ptr(slots), _stream(stream)))


def moe_decode_workspace_bytes(shape) -> int:
    return load().moe_decode_workspace_bytes(ctypes.byref(shape))


def moe_decode(shape, layer, x, norm_eps, slots, weights, codebook, y, accumulate, ctrl, ws, ws_bytes, stream=None):
    _check("moe_decode", load().moe_decode(ctypes.byref(shape), layer, ptr(x), float(norm_eps), ptr(slots), ptr(weights),
                                           ptr(codebook), ptr(y), int(accumulate), ptr(ctrl), ptr(ws), ws_bytes,
                                           _stream(stream)))


def moe_decode_static(shape, layer, x, norm_eps, slots, weights, codebook, y, accumulate, ctrl, stream=None):
    _check("moe_decode_static", load().moe_decode_static(ctypes.byref(shape), layer, ptr(x), float(norm_eps),
                                                         ptr(slots), ptr(weights), ptr(codebook), ptr(y),
                                                         int(accumulate), ptr(ctrl), _stream(stream)))


def moe_decode_stack_workspace_bytes(shape) -> int:
    return load().moe_decode_stack_workspace_bytes(ctypes.byref(shape))


def moe_decode_stack(shape, layer0, n_layers, x, norm_eps, w_router, bias, residency, codebook, ids, weights, slots,
                     miss, ctrl, logits_out, x_hist, pregate, pregate_hits, ws, ws_bytes, stream=None):
    _check("moe_decode_stack", load().moe_decode_stack(
        ctypes.byref(shape), layer0, n_layers, ptr(x), float(norm_eps), ptr(w_router), ptr(bias), ptr(residency),
        ptr(codebook), ptr(ids), ptr(weights), ptr(slots), ptr(miss), ptr(ctrl), ptr(logits_out), ptr(x_hist),
        int(pregate), ptr(pregate_hits), ptr(ws), ws_bytes, _stream(stream)))


def moe_decode_stack_fill(shape, layer0, n_layers, x, norm_eps, w_router, bias, residency, codebook, ids, weights,
                          slots, miss, ctrl, logits_out, x_hist, fill_src, fill_dst, filled, ws, ws_bytes, stream=None):
    _check("moe_decode_stack_fill", load().moe_decode_stack_fill(
        ctypes.byref(shape), layer0, n_layers, ptr(x), float(norm_eps), ptr(w_router), ptr(bias), ptr(residency),
        ptr(codebook), ptr(ids), ptr(weights), ptr(slots), ptr(miss), ptr(ctrl), ptr(logits_out), ptr(x_hist),
        ptr(fill_src), ptr(fill_dst), ptr(filled), ptr(ws), ws_bytes, _stream(stream)))


def moe_decode_layer(shape, layer, x, norm_eps, w_router, bias, residency, codebook, ids, weights, slots, miss, ctrl,
                     logits_out, y, ws, ws_bytes, stream=None):
    _check("moe_decode_layer", load().moe_decode_layer(
        ctypes.byref(shape), layer, ptr(x), float(norm_eps), ptr(w_router), ptr(bias), ptr(residency), ptr(codebook),
        ptr(ids), ptr(weights), ptr(slots), ptr(miss), ptr(ctrl), ptr(logits_out), ptr(y), ptr(ws), ws_bytes,
        _stream(stream)))


_dtypes = None


def _typed(what: str, t, allowed, numel: int | None = None) -> int:
    """RL_* code of a tensor's type; refuses other types than `allowed` and, with `numel`, other
    sizes (the library only sees an address)."""
    global _dtypes
    if _dtypes is None:
        import torch
        _dtypes = {torch.float32: RL_F32, torch.float16: RL_F16, torch.bfloat16: RL_BF16,
                   torch.float8_e4m3fn: RL_F8_E4M3}
    code = _dtypes.get(t.dtype, -1)
    if code not in allowed:
        raise ValueError(f"{what}: a tensor of type {t.dtype} is not supported here")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{what}: {numel} values expected, got shape {tuple(t.shape)}")
    return code


_kinds = None


def _load_kinds():
    """What the tensor types of a buffer may be.  Integers may come signed or unsigned (torch has few
    operations on unsigned ones), 8-bit floats also as their bytes."""
    global _kinds
    import torch
    u = lambda n: tuple(getattr(torch, k) for k in (f"int{n}", f"uint{n}") if hasattr(torch, k))  # noqa: E731
    _kinds = {"f32": (torch.float32,), "i32": u(32), "i64": u(64), "bytes": u(8),
              "e4m3": (torch.float8_e4m3fn, *u(8))}
    return _kinds


def _sized(what: str, t, kind: str, numel: int) -> None:
    """Refuses a buffer of another type or of another size than the call's."""
    if t is not None and (t.dtype not in (_kinds or _load_kinds())[kind] or t.numel() != numel):
        raise ValueError(f"{what}: {numel} items of type {kind} expected, got {t.dtype} {tuple(t.shape)}")


def _holds(what: str, t, kind: str, numel: int) -> None:
    """Refuses a buffer of another type or of fewer items than a call reads or writes."""
    if t is not None and (t.dtype not in (_kinds or _load_kinds())[kind] or t.numel() < numel):
        raise ValueError(f"{what}: {numel} items of type {kind} needed, got {t.dtype} {tuple(t.shape)}")


def _ptrs(*tensors):
    """Raw addresses of device tensors (None: NULL), all dense and on the current device, where the
    call will launch."""
    device = (_current or _cuda())[0]()
    out = []
    for t in tensors:
        if t is None:
            out.append(None)
        elif t.get_device() != device:
            raise ValueError(f"tensor on {t.device} passed to a call on cuda:{device}")
        elif not t.is_contiguous():
            raise ValueError(f"tensor of shape {tuple(t.shape)} and strides {t.stride()} is not contiguous")
        else:
            out.append(t.data_ptr())
    return out


_ROW = (RL_F32, RL_F16, RL_BF16)


def moe_decode_tokens_workspace_bytes(shape, T) -> int:
    return load().moe_decode_tokens_workspace_bytes(ctypes.byref(shape), T)


def moe_decode_tokens(shape, layer, T, x, norm_eps, w_router, bias, residency, codebook, ids, weights, slots, miss,
                      ctrl, logits_out, y, accumulate, ws, ws_bytes, stream=None):
    H, E, TK, layers = shape.hidden, shape.n_experts, T * shape.top_k, shape.n_layers
    _holds("x", x, "f32", T * H)
    _holds("w_router", w_router, "f32", E * H)
    _holds("bias", bias, "f32", E)
    _holds("residency", residency, "i64", layers * E)
    _holds("codebook", codebook, "bytes", 2048)
    _holds("ids", ids, "i32", TK)
    _holds("weights", weights, "f32", TK)
    _holds("slots", slots, "i64", TK)
    _holds("miss", miss, "i32", layers)
    _holds("ctrl", ctrl, "i32", 2)
    _holds("logits_out", logits_out, "f32", T * E)
    _holds("y", y, "f32", T * H)
    _holds("ws", ws, "bytes", ws_bytes)
    x, w, bias, res, cb, ids, wt, slots, miss, ctrl, lg, y, ws = _ptrs(x, w_router, bias, residency, codebook, ids,
                                                                       weights, slots, miss, ctrl, logits_out, y, ws)
    _check("moe_decode_tokens", load().moe_decode_tokens(
        ctypes.byref(shape), layer, T, x, norm_eps, w, bias, res, cb, ids, wt, slots, miss, ctrl, lg, y,
        int(accumulate), ws, ws_bytes, _stream(stream)))


def rl_add_rmsnorm(x, T, H, eps, res=None, gain=None, x_out=None, xn=None, q=None, scale=None, group=128, stream=None):
    """x (+ res) -> x_out, RMSNorm (* gain) -> xn and, in 8 bits with group scales, (q, scale); any output
    may be None.  The row type is x's."""
    n = T * H
    dt = _typed("x", x, _ROW, n)
    for what, t in (("res", res), ("x_out", x_out), ("xn", xn)):
        if t is not None and (t.dtype != x.dtype or t.numel() != n):
            raise ValueError(f"{what}: {n} values of {x.dtype} expected, got {t.dtype} {tuple(t.shape)}")
    if gain is not None:
        _typed("gain", gain, (RL_F32,), H)
    if q is not None:
        _sized("q", q, "e4m3", n)
    if scale is not None and group > 0:
        _typed("scale", scale, (RL_F32,), T * (H // group))
    x, res, gain, x_out, xn, q, scale = _ptrs(x, res, gain, x_out, xn, q, scale)
    _check("rl_add_rmsnorm", load().rl_add_rmsnorm(x, res, gain, dt, T, H, eps, x_out, xn, q, scale, group,
                                                   _stream(stream)))


def rl_q4_matvec(w, w_scale, x, y, T, N, K, group, x_scale=None, accumulate=0, stream=None):
    """y [T][N] (+)= x [T][K] times the 4-bit matrix (w, w_scale) transposed; types from the tensors, x in
    e4m3 with x_scale [T][K / group]."""
    xdt, ydt = _typed("x", x, (*_ROW, RL_F8_E4M3), T * K), _typed("y", y, _ROW, T * N)
    _sized("w", w, "bytes", N * K // 2)
    if group > 0:
        _typed("w_scale", w_scale, (RL_F16,), N * (K // group))
        if x_scale is not None:
            _typed("x_scale", x_scale, (RL_F32,), T * (K // group))
    w, w_scale, x, x_scale, y = _ptrs(w, w_scale, x, x_scale, y)
    _check("rl_q4_matvec", load().rl_q4_matvec(w, w_scale, N, K, group, x, xdt, x_scale, T, y, ydt, accumulate,
                                               _stream(stream)))


def _blocks(n: int) -> int:
    return -(-n // 128)


def rl_f8_matmul(w, w_scale, x, x_scale, y, T, N, K, res=None, layer=0, ctrl=None, stream=None):
    """y [T][N] = (res +) x [T][K] times w [N][K] transposed, both e4m3 with a scale per block of 128; y's type
    is the tensor's.  With ctrl, nothing where layer `layer` or an earlier one raised the flag."""
    dt = _typed("y", y, _ROW, T * N)
    if res is not None and (res.dtype != y.dtype or res.numel() != T * N):
        raise ValueError(f"res: {T * N} values of {y.dtype} expected, got {res.dtype} {tuple(res.shape)}")
    _sized("w", w, "e4m3", N * K)
    _sized("w_scale", w_scale, "f32", _blocks(N) * _blocks(K))
    _sized("x", x, "e4m3", T * K)
    _sized("x_scale", x_scale, "f32", T * _blocks(K))
    _holds("ctrl", ctrl, "i32", 2)
    w, w_scale, x, x_scale, res, y, ctrl = _ptrs(w, w_scale, x, x_scale, res, y, ctrl)
    _check("rl_f8_matmul", load().rl_f8_matmul(w, w_scale, N, K, x, x_scale, T, res, y, dt, layer, ctrl, _stream(stream)))


def rl_f8_gated(w_gate, gate_scale, w_up, up_scale, x, x_scale, T, I, K, h=None, q=None, scale=None, layer=0, ctrl=None,
                stream=None):
    """silu(x w_gate^T) * (x w_up^T) for rows x [T][K], all e4m3 with a scale per block of 128, into h [T][I] of
    its tensor's type or in 8 bits (q, scale), or both."""
    dt = RL_F32 if h is None else _typed("h", h, _ROW, T * I)
    for what, t, kind, n in (("w_gate", w_gate, "e4m3", I * K), ("gate_scale", gate_scale, "f32", _blocks(I) * _blocks(K)),
                             ("w_up", w_up, "e4m3", I * K), ("up_scale", up_scale, "f32", _blocks(I) * _blocks(K)),
                             ("x", x, "e4m3", T * K), ("x_scale", x_scale, "f32", T * _blocks(K)),
                             ("q", q, "e4m3", T * I), ("scale", scale, "f32", T * _blocks(I))):
        _sized(what, t, kind, n)
    _holds("ctrl", ctrl, "i32", 2)
    w_gate, gate_scale, w_up, up_scale, x, x_scale, h, q, scale, ctrl = _ptrs(w_gate, gate_scale, w_up, up_scale, x, x_scale,
                                                                             h, q, scale, ctrl)
    _check("rl_f8_gated", load().rl_f8_gated(w_gate, gate_scale, w_up, up_scale, I, K, x, x_scale, T, h, dt, q, scale, layer,
                                             ctrl, _stream(stream)))


def rl_logprobs_workspace_bytes(T, V, top_n) -> int:
    return load().rl_logprobs_workspace_bytes(T, V, top_n)


def rl_logprobs(logits, T, V, targets, logprob, entropy, top_n, top_ids, top_logprob, ws, ws_bytes, stream=None):
    dt = _typed("logits", logits, _ROW, T * V)
    _sized("targets", targets, "i32", T)
    _sized("logprob", logprob, "f32", T)
    _sized("entropy", entropy, "f32", T)
    _sized("top_ids", top_ids, "i32", T * top_n)
    _sized("top_logprob", top_logprob, "f32", T * top_n)
    _holds("ws", ws, "bytes", ws_bytes)
    x, targets, logprob, entropy, ids, top, ws = _ptrs(logits, targets, logprob, entropy, top_ids, top_logprob, ws)
    _check("rl_logprobs", load().rl_logprobs(x, dt, T, V, targets, logprob, entropy, top_n, ids, top, ws, ws_bytes,
                                             _stream(stream)))


def rl_sample(logits, T, V, uniform, ids, temperature=None, top_k=None, top_p=None, min_p=None, logprob=None, stream=None):
    """The next token of each row of logits [T][V] into ids (int32 [T]), drawn by uniform (f32 [T]); one temperature,
    top_k (int32), top_p and min_p per row, each may be None."""
    dt = _typed("logits", logits, _ROW, T * V)
    for what, t, kind in (("uniform", uniform, "f32"), ("ids", ids, "i32"), ("temperature", temperature, "f32"),
                          ("top_k", top_k, "i32"), ("top_p", top_p, "f32"), ("min_p", min_p, "f32"),
                          ("logprob", logprob, "f32")):
        _sized(what, t, kind, T)
    x, u, temp, k, p, m, ids, lp = _ptrs(logits, uniform, temperature, top_k, top_p, min_p, ids, logprob)
    _check("rl_sample", load().rl_sample(x, dt, T, V, u, temp, k, p, m, ids, lp, _stream(stream)))


def rl_build_pairs_workspace_bytes(shape, T) -> int:
    return load().rl_build_pairs_workspace_bytes(ctypes.byref(shape), T)


def rl_build_pairs(shape, layer, T, ids, offs, pair_tok, pair_k, ctrl, ws=None, ws_bytes=0, stream=None):
    _check("rl_build_pairs", load().rl_build_pairs(ctypes.byref(shape), layer, T, ptr(ids), ptr(offs),
                                                   ptr(pair_tok), ptr(pair_k), ptr(ctrl), ptr(ws), ws_bytes,
                                                   _stream(stream)))


def moe_prefill_workspace_bytes(shape, T) -> int:
    return load().moe_prefill_workspace_bytes(ctypes.byref(shape), T)


def moe_prefill_chunk(shape, layer, T, xn, offs, pair_tok, pair_k, slots, weights, codebook, y, accumulate,
                      ctrl, ws, ws_bytes, stream=None):
    _check("moe_prefill_chunk", load().moe_prefill_chunk(
        ctypes.byref(shape), layer, T, ptr(xn), ptr(offs), ptr(pair_tok), ptr(pair_k), ptr(slots), ptr(weights),
        ptr(codebook), ptr(y), int(accumulate), ptr(ctrl), ptr(ws), ws_bytes, _stream(stream)))


def moe_prefill_chunk_f32(shape, layer, T, xn, offs, pair_tok, pair_k, slots, weights, codebook, y, accumulate,
                          ctrl, ws, ws_bytes, stream=None):
    _check("moe_prefill_chunk_f32", load().moe_prefill_chunk_f32(
        ctypes.byref(shape), layer, T, ptr(xn), ptr(offs), ptr(pair_tok), ptr(pair_k), ptr(slots), ptr(weights),
        ptr(codebook), ptr(y), int(accumulate), ptr(ctrl), ptr(ws), ws_bytes, _stream(stream)))
