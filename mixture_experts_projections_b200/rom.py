"""Python binding of librom.so (the C ABI in include/rom.h).

Argument marshalling only: every step of the RoM block runs in the CUDA
library. PyTorch supplies device memory and the current stream. The functions
keep the C names (rom_route, rom_dispatch, rom_expert_proj, rom_combine, ...);
``block_forward`` and ``inproj_forward`` chain them for one block.

Importing this module does not need a GPU; calling into the library does, and
a missing library raises at once (there is no fallback path).
"""
from __future__ import annotations

import ctypes
import os
import warnings

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "librom.so")

ROM_OK, ROM_ERR_INVALID_ARG, ROM_ERR_UNSUPPORTED, ROM_ERR_WORKSPACE, ROM_ERR_CUDA, \
    ROM_ERR_TIMEOUT, ROM_ERR_ROUTING = range(7)
ROM_F32, ROM_BF16 = 0, 1
ROM_PROJ_CONV_GATE, ROM_PROJ_OUT, ROM_PROJ_INPROJ, ROM_PROJ_SLOTS, ROM_PROJ_CONV_GATE_SLOTS = \
    0, 1, 2, 3, 4
ROM_COMBINE_SUM, ROM_COMBINE_GATE, ROM_COMBINE_GATE_DENSE = 0, 1, 2
ROM_W_TILED = 0x100  # rom_expert_proj_dense: weights in the tile-major layout

# Every exported symbol of include/rom.h with its ctypes signature.
_P = ctypes.c_void_p
_I = ctypes.c_int
_L = ctypes.c_int64
SIGNATURES = {
    "rom_status_string": (ctypes.c_char_p, [_I]),
    "rom_version": (_I, []),
    "rom_workspace_size": (ctypes.c_size_t, [_L, _I]),
    "rom_route": (_I, [_P, _I, _L, _I, _P, _P, _I, _I, _I, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "rom_dispatch": (_I, [_P, _I, _L, _I, _I, _I, _P, _P, ctypes.c_size_t, _P, _P, _P, _P, _P]),
    "rom_expert_proj": (_I, [_I, _I, _P, _L, _I, _P, _P, _I, _I, _I, _P, _P, _P, _P, _P]),
    "rom_combine": (_I, [_I, _I, _P, _L, _I, _I, _P, _P, _P]),
    "rom_expert_proj_dense": (_I, [_I, _I, _P, _L, _I, _P, _I, _I, _I, _P, _P, _P, _P]),
    "rom_pack_expert_weights": (_I, [_I, _P, _I, _I, _I, _P, _P]),
    "rom_get_status": (_I, [_P, ctypes.POINTER(ctypes.c_int32)]),
    "rom_debug_wait_timeout": (_I, [ctypes.c_uint64, _P]),
    "rom_route_dispatch_noalloc": (_I, [_P, _I, _L, _I, _P, _P, _I, _I, _I, _P, _P, _P, _P, _P,
                                        _P, _P, _P]),
    "rom_bwd_gather": (_I, [_P, _L, _I, _I, _P, _P, _P, _P]),
    "rom_bwd_dgrad_out": (_I, [_P, _L, _I, _P, _I, _I, _I, _P, _P, _P, _P, _P, _P]),
    "rom_bwd_gate": (_I, [_P, _P, _L, _I, _I, _P, _P, _P]),
    "rom_bwd_dgrad_in": (_I, [_P, _L, _I, _P, _P, _I, _I, _I, _P, _P, _P, _P]),
    "rom_route_bwd": (_I, [_L, _I, _I, _I, _I, _P, _P, _P, _P, _I, _P, _P, _P, _P, _P]),
    "rom_route_probs": (_I, [_P, _I, _L, _I, _P, _P, _I, _P, _P]),
    "rom_route_wgrad": (_I, [_P, _I, _L, _I, _I, _P, _P, _P, _P]),
    "rom_bwd_wgrad": (_I, [_P, _I, _P, _I, _L, _I, _P, _I, _P, _P, _P]),
    "rom_ssm_core_workspace_size": (ctypes.c_size_t, [_L, _I, _I, _I, _I, _I]),
    "rom_ssm_core_routed_workspace_size": (ctypes.c_size_t, [_L, _I, _I, _I, _I, _I, _I, _I]),
    "rom_ssm_core_routed": (_I, [_P, _L, _I, _I, _P, _P, _I, _P, _I, _I, _I, _P, _P, _P, _P,
                                 _I, _I, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "rom_ssm_core": (_I, [_P, _L, _I, _I, _P, _P, _I, _P, _I, _I, _I, _P, _P, _P, _P, _P, _P,
                          ctypes.c_size_t, _P]),
    "rom_add_rmsnorm": (_I, [_P, _I, _P, _I, _L, _I, _P, ctypes.c_float, _P, _P, _P, _P, _P, _P]),
    "rom_add_rmsnorm_bwd_workspace_size": (ctypes.c_size_t, [_L, _I]),
    "rom_add_rmsnorm_bwd": (_I, [_P, _I, _P, _P, _I, _L, _I, _P, _P, _P, _P, _P, _P,
                                 ctypes.c_size_t, _P]),
    "rom_quant_rows": (_I, [_P, _I, _L, _I, _P, _P, _P]),
    "rom_dispatch_q8": (_I, [_P, _P, _L, _I, _I, _I, _P, _P, ctypes.c_size_t, _P, _P, _P, _P, _P,
                             _P]),
    "rom_expert_proj_q8": (_I, [_I, _P, _P, _L, _I, _P, _P, _P, _P, _I, _I, _I, _P, _P, _P, _P,
                                _P]),
    "rom_w4_code_bytes": (ctypes.c_size_t, [_I, _I, _I]),
    "rom_w4_scale_bytes": (ctypes.c_size_t, [_I, _I, _I, _I]),
    "rom_quant_expert_weights_w4": (_I, [_I, _P, _I, _I, _I, _I, _P, _P, _P]),
    "rom_expert_proj_w4": (_I, [_I, _P, _L, _I, _P, _P, _P, _P, _I, _I, _I, _I, _P, _P, _P, _P]),
}

_lib = None
# binding/fast_calls.cpp, once the library is loaded (None where it is not built or
# does not load: the calls below then check their tensors in Python, at 0.4 us each).
_fast = None
_FAST_CALLS = ("rom_add_rmsnorm", "rom_add_rmsnorm_bwd", "rom_quant_rows", "rom_expert_proj_q8",
               "rom_expert_proj_w4")


class RomError(RuntimeError):
    pass


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load librom.so (once) and declare the signatures of its entry points."""
    global _lib
    if _lib is None:
        if not os.path.exists(path):
            raise RomError(f"{path} is missing: build it with "
                           "`python -m mixture_experts_projections_b200.build`")
        lib = ctypes.CDLL(path)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
        if path == LIB_PATH and os.path.exists(os.path.join(_HERE, "_fast_calls.so")):
            try:
                _load_fast_calls(lib)
            except (ImportError, OSError) as e:
                warnings.warn(f"{e}: tensors are checked in Python, a few microseconds per call "
                              "more", RuntimeWarning, stacklevel=2)
    return _lib


def _load_fast_calls(lib):
    global _fast
    from . import _fast_calls
    built = getattr(_fast_calls, "torch_version", "unknown")
    if not torch.__version__.startswith(built):
        raise ImportError(f"_fast_calls.so was built against torch {built}, this is "
                          f"{torch.__version__}")
    _fast_calls.bind(*(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in _FAST_CALLS))
    _fast = _fast_calls


def _fast_done(code, fn):
    """Whether a call of _fast was made (it returns None where its arguments are
    not what it takes); raises its error."""
    if code is None:
        return False
    if code != ROM_OK:
        _check(code, fn)
    return True


def _check(code: int, what: str):
    if code != ROM_OK:
        msg = load_library().rom_status_string(code).decode()
        raise RomError(f"{what} failed: {msg} ({code})")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return ROM_BF16
    if t.dtype == torch.float32:
        return ROM_F32
    raise RomError(f"unsupported dtype {t.dtype}")


def _need(t: torch.Tensor, name: str):
    if not t.is_cuda or not t.is_contiguous():
        raise RomError(f"{name} must be a contiguous CUDA tensor")


# ------------------------------------------------------------------ C entry points


def rom_workspace_size(T: int, E: int) -> int:
    return int(load_library().rom_workspace_size(T, E))


def rom_route(x, w_r, bias, k, renorm, topk_idx, topk_w, counts, ws, stream=None):
    for t, n in ((x, "x"), (w_r, "w_r"), (topk_idx, "topk_idx"), (topk_w, "topk_w")):
        _need(t, n)
    T, Dm = x.shape
    E = w_r.shape[1]
    _check(load_library().rom_route(
        _ptr(x), _dtype_code(x), T, Dm, _ptr(w_r), _ptr(bias), E, k, int(renorm),
        _ptr(topk_idx), _ptr(topk_w), _ptr(counts), _ptr(ws),
        0 if ws is None else ws.numel() * ws.element_size(), _stream(stream)), "rom_route")


def rom_dispatch(x, E, k, topk_idx, ws, offsets, sorted_slot, slot_pos, x_sorted, stream=None):
    T, Dm = x.shape
    _check(load_library().rom_dispatch(
        _ptr(x), _dtype_code(x), T, Dm, E, k, _ptr(topk_idx), _ptr(ws),
        0 if ws is None else ws.numel() * ws.element_size(), _ptr(offsets), _ptr(sorted_slot),
        _ptr(slot_pos), _ptr(x_sorted), _stream(stream)), "rom_dispatch")


def rom_expert_proj(proj, a_sorted, w0, w1, E, k, offsets, sorted_slot, topk_w, out,
                    stream=None):
    R, K = a_sorted.shape
    N = w0.shape[1]
    if not out.is_contiguous():
        raise RomError("out must be contiguous")
    _check(load_library().rom_expert_proj(
        proj, _dtype_code(a_sorted), _ptr(a_sorted), R, K, _ptr(w0), _ptr(w1), N, E, k,
        _ptr(offsets), _ptr(sorted_slot), _ptr(topk_w), _ptr(out), _stream(stream)),
        "rom_expert_proj")


def rom_expert_proj_dense(proj, x, w, E, k, topk_idx, topk_w, out, stream=None, tiled=False):
    """``tiled``: ``w`` holds the weights in the tile-major layout of
    pack_expert_weights (the same [E, N, K] shape and values, stored by tile)."""
    T, K = x.shape
    N = w.shape[1]
    _check(load_library().rom_expert_proj_dense(
        proj | (ROM_W_TILED if tiled else 0), _dtype_code(x), _ptr(x), T, K, _ptr(w), N, E, k,
        _ptr(topk_idx), _ptr(topk_w), _ptr(out), _stream(stream)), "rom_expert_proj_dense")


def pack_expert_weights(w, stream=None):
    """A copy of the expert weights w [E, N, K] (bf16) in the tile-major layout
    (each 128 x 64 weight tile one contiguous 16 KB block) that
    rom_expert_proj_dense reads with ``tiled=True``. Returned with the shape
    [E, N, K]; its elements are in tile order, not row order."""
    _need(w, "w")
    E, N, K = w.shape
    out = torch.empty_like(w)
    _check(load_library().rom_pack_expert_weights(_dtype_code(w), _ptr(w), E, N, K, _ptr(out),
                                                  _stream(stream)), "rom_pack_expert_weights")
    return out


# Few tokens: the routed projection reads x in token order and needs no
# dispatch (rom_expert_proj_dense).
DENSE_SMALL_MAX_TOKENS = 64


def rom_combine(mode, dtype_code, inp, T, k, N, slot_pos, out, stream=None):
    _check(load_library().rom_combine(mode, dtype_code, _ptr(inp), T, k, N, _ptr(slot_pos),
                                      _ptr(out), _stream(stream)), "rom_combine")


def rom_get_status(stream=None) -> int:
    v = ctypes.c_int32(0)
    _check(load_library().rom_get_status(_stream(stream), ctypes.byref(v)), "rom_get_status")
    return int(v.value)


def rom_debug_wait_timeout(limit_ns: int, stream=None):
    _check(load_library().rom_debug_wait_timeout(limit_ns, _stream(stream)),
           "rom_debug_wait_timeout")


def rom_route_dispatch_noalloc(x, w_r, bias, k, renorm, topk_idx, topk_w, counts, offsets,
                               sorted_slot, slot_pos, x_sorted, stream=None):
    """Routing + dispatch without a caller workspace (the library's own fixed
    device scratch; see include/rom.h)."""
    T, Dm = x.shape
    E = w_r.shape[1]
    _check(load_library().rom_route_dispatch_noalloc(
        _ptr(x), _dtype_code(x), T, Dm, _ptr(w_r), _ptr(bias), E, k, int(renorm),
        _ptr(topk_idx), _ptr(topk_w), _ptr(counts), _ptr(offsets), _ptr(sorted_slot),
        _ptr(slot_pos), _ptr(x_sorted), _stream(stream)), "rom_route_dispatch_noalloc")


# ------------------------------------------------------------------ norm, 8-bit and 4-bit data
#
# These entry points check every tensor (type, shape, contiguity, one device)
# before the library is called, run on the tensors' device whichever device is
# current, and take the current stream of that device unless given one.


def _t(t, name, dtype, shape, dev):
    """Refuses a tensor of another type, shape, layout or device than cuda:dev;
    returns its address."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        if t.dtype is not dtype or t.shape != shape:
            raise RomError(f"{name} must be {dtype} {list(shape)}, got {t.dtype} {list(t.shape)}")
        if not t.is_cuda or not t.is_contiguous():
            raise RomError(f"{name} must be a contiguous CUDA tensor")
        raise RomError(f"{name} is on {t.device}, the call's first tensor on cuda:{dev}")
    return t.data_ptr()


def _device(t, name):
    """The index of the CUDA device that a call runs on: that of its first tensor."""
    dev = t.get_device()
    if dev < 0:
        raise RomError(f"{name} must be a contiguous CUDA tensor")
    return dev


def _ws(t, dev):
    """Address and bytes of a workspace (or None)."""
    if t is None:
        return None, 0
    if t.get_device() != dev or not t.is_contiguous():
        raise RomError(f"ws must be a contiguous tensor on cuda:{dev}")
    return t.data_ptr(), t.numel() * t.element_size()


def _call(fn, dev, stream, *args):
    """Calls a library function with the stream as its last argument, on device
    ``dev`` and its current stream unless one is given."""
    if stream is None:
        # the handle alone: a Stream object costs 1.2 us of a 9 us call
        handle = torch._C._cuda_getCurrentRawStream(dev)
    elif stream.device.index == dev:
        handle = stream.cuda_stream
    else:
        raise RomError(f"{fn}: the stream is not one of cuda:{dev}")
    f = getattr(_lib or load_library(), fn)
    if torch.cuda.current_device() == dev:
        code = f(*args, handle)
    else:
        with torch.cuda.device(dev):
            code = f(*args, handle)
    if code != ROM_OK:
        _check(code, fn)


_BF16, _F32, _I32, _E4M3 = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn


def rom_add_rmsnorm(x, residual, weight, eps, res_out, y, y8=None, y_scale=None, rstd=None,
                    stream=None):
    """s = x + residual (to ``res_out``, may be ``residual``), y = s * rstd *
    weight with rstd = 1 / sqrt(mean s^2 + eps), per row of [T, Dm]. Any of the
    outputs may be None; ``y8`` (e4m3) and ``y_scale`` come together. The
    residual stream's type is that of ``residual`` or ``res_out``."""
    if stream is None and _fast is not None and _fast_done(
            _fast.add_rmsnorm(x, residual, weight, eps, res_out, y, y8, y_scale, rstd),
            "rom_add_rmsnorm"):
        return
    T, D = x.shape
    rt = residual.dtype if residual is not None else (res_out.dtype if res_out is not None else _F32)
    code = _dtype_code(x)
    dev = _device(x, "x")
    _call("rom_add_rmsnorm", dev, stream, _t(x, "x", x.dtype, (T, D), dev), code,
          None if residual is None else _t(residual, "residual", rt, (T, D), dev),
          ROM_BF16 if rt is _BF16 else ROM_F32 if rt is _F32 else -1, T, D,
          _t(weight, "weight", _F32, (D,), dev), eps,
          None if res_out is None else _t(res_out, "res_out", rt, (T, D), dev),
          None if y is None else _t(y, "y", x.dtype, (T, D), dev),
          None if y8 is None else _t(y8, "y8", _E4M3, (T, D), dev),
          None if y_scale is None else _t(y_scale, "y_scale", _F32, (T,), dev),
          None if rstd is None else _t(rstd, "rstd", _F32, (T,), dev))


def rom_add_rmsnorm_bwd_workspace_size(T: int, D: int) -> int:
    return int(load_library().rom_add_rmsnorm_bwd_workspace_size(T, D))


def rom_add_rmsnorm_bwd(dy, dres_out, res_out, weight, rstd, dx, dres, dw, ws, stream=None):
    """Gradient of rom_add_rmsnorm: dx (type of dy) and dres (type of res_out,
    may be ``dres_out``) are the same values, dw float32 [Dm]; each may be
    None, and so may ``dres_out``. ``ws``: at least
    rom_add_rmsnorm_bwd_workspace_size(T, Dm) bytes, for dw."""
    if stream is None and _fast is not None and _fast_done(
            _fast.add_rmsnorm_bwd(dy, dres_out, res_out, weight, rstd, dx, dres, dw, ws),
            "rom_add_rmsnorm_bwd"):
        return
    T, D = dy.shape
    rt = res_out.dtype
    code = _dtype_code(dy)
    dev = _device(dy, "dy")
    _call("rom_add_rmsnorm_bwd", dev, stream, _t(dy, "dy", dy.dtype, (T, D), dev), code,
          None if dres_out is None else _t(dres_out, "dres_out", rt, (T, D), dev),
          _t(res_out, "res_out", rt, (T, D), dev),
          ROM_BF16 if rt is _BF16 else ROM_F32 if rt is _F32 else -1, T, D,
          _t(weight, "weight", _F32, (D,), dev), _t(rstd, "rstd", _F32, (T,), dev),
          None if dx is None else _t(dx, "dx", dy.dtype, (T, D), dev),
          None if dres is None else _t(dres, "dres", rt, (T, D), dev),
          None if dw is None else _t(dw, "dw", _F32, (D,), dev), *_ws(ws, dev))


def rom_quant_rows(x, q, scale, stream=None):
    """The rows of x [rows, K] as e4m3 codes ``q`` and a float32 scale each."""
    if stream is None and _fast is not None and _fast_done(_fast.quant_rows(x, q, scale),
                                                           "rom_quant_rows"):
        return
    rows, K = x.shape
    code = _dtype_code(x)
    dev = _device(x, "x")
    _call("rom_quant_rows", dev, stream, _t(x, "x", x.dtype, (rows, K), dev), code, rows, K,
          _t(q, "q", _E4M3, (rows, K), dev), _t(scale, "scale", _F32, (rows,), dev))


def rom_dispatch_q8(x8, x_scale, E, k, topk_idx, ws, offsets, sorted_slot, slot_pos, x8_sorted,
                    scale_sorted, stream=None):
    T, D = x8.shape
    R = T * k
    n = max(R, 1)
    dev = _device(x8, "x8")
    _call("rom_dispatch_q8", dev, stream, _t(x8, "x8", _E4M3, (T, D), dev),
          _t(x_scale, "x_scale", _F32, (T,), dev), T, D, E, k,
          _t(topk_idx, "topk_idx", _I32, (T, k), dev), *_ws(ws, dev),
          _t(offsets, "offsets", _I32, (E + 1,), dev),
          _t(sorted_slot, "sorted_slot", _I32, (n,), dev),
          _t(slot_pos, "slot_pos", _I32, (n,), dev),
          _t(x8_sorted, "x8_sorted", _E4M3, (n, D), dev),
          _t(scale_sorted, "scale_sorted", _F32, (n,), dev))


def rom_expert_proj_q8(proj, a_sorted, a_scale, w0, w0_scale, w1, w1_scale, k, offsets,
                       sorted_slot, topk_w, out, stream=None):
    """rom_expert_proj on e4m3 rows [R, K] and weights [E, N, K] with float32
    scales [R] and [E, N]. ``out`` as there, in bf16 or (slot rows) float32."""
    if stream is None and _fast is not None and _fast_done(
            _fast.expert_proj_q8(proj, a_sorted, a_scale, w0, w0_scale, w1, w1_scale, k, offsets,
                                 sorted_slot, topk_w, out), "rom_expert_proj_q8"):
        return
    R, K = a_sorted.shape
    E, N, _ = w0.shape
    dev = _device(a_sorted, "a_sorted")
    gate = proj == ROM_PROJ_CONV_GATE or proj == ROM_PROJ_CONV_GATE_SLOTS
    if gate and (w1 is None or w1_scale is None):
        raise RomError("the Conv+Gate projections need w1 and w1_scale")
    if k < 1 or R % k:
        raise RomError(f"{R} rows are no multiple of k = {k}")
    if k == 1 and (proj == ROM_PROJ_OUT or proj == ROM_PROJ_INPROJ or proj == ROM_PROJ_CONV_GATE):
        po = _t(out, "out", _BF16, (R, N), dev)
    else:
        shape = (2, R, N) if gate else (R, N)
        po = _t(out, "out", _F32, shape, dev)
    if sorted_slot is not None and sorted_slot.shape[0] < R:
        raise RomError(f"sorted_slot must hold {R} slots")
    if topk_w is not None and topk_w.numel() != R:
        raise RomError(f"topk_w must hold {R} weights")
    _call("rom_expert_proj_q8", dev, stream, proj, _t(a_sorted, "a_sorted", _E4M3, (R, K), dev),
          _t(a_scale, "a_scale", _F32, (R,), dev), R, K, _t(w0, "w0", _E4M3, (E, N, K), dev),
          _t(w0_scale, "w0_scale", _F32, (E, N), dev),
          _t(w1, "w1", _E4M3, (E, N, K), dev) if gate else None,
          _t(w1_scale, "w1_scale", _F32, (E, N), dev) if gate else None, N, E, k,
          None if offsets is None else _t(offsets, "offsets", _I32, (E + 1,), dev),
          None if sorted_slot is None else _t(sorted_slot, "sorted_slot", _I32,
                                              (sorted_slot.shape[0],), dev),
          None if topk_w is None else _t(topk_w, "topk_w", _F32, topk_w.shape, dev), po)


def rom_quant_expert_weights_w4(w, group, q, s, stream=None):
    """w [E, N, K] (bf16 or float32) to 4-bit codes ``q`` uint8 [E, Nt, Kb, 2, 8,
    4, 16] and bf16 scales ``s`` [E, Nt, Kb, 16, 128 / group] (Nt = ceil(N / 16),
    Kb = ceil(K / 128); the layout is in include/rom.h)."""
    E, N, K = w.shape
    if group not in (32, 64, 128):
        raise RomError(f"group must be 32, 64 or 128, got {group}")
    nt, kb = -(-N // 16), -(-K // 128)
    code = _dtype_code(w)
    dev = _device(w, "w")
    _call("rom_quant_expert_weights_w4", dev, stream, code, _t(w, "w", w.dtype, (E, N, K), dev), E,
          N, K, group, _t(q, "q", torch.uint8, (E, nt, kb, 2, 8, 4, 16), dev),
          _t(s, "s", _BF16, (E, nt, kb, 16, 128 // group), dev))


def rom_expert_proj_w4(proj, x, q0, s0, q1, s1, N, k, topk_idx, topk_w, out, stream=None):
    """Routed projection of T <= 64 tokens x [T, K] (bf16) on 4-bit weights, in
    token order without a dispatch. ROM_PROJ_OUT and ROM_PROJ_INPROJ: weighted,
    out bf16 [T, N] (k == 1) or float32 [T*k, N]; ROM_PROJ_SLOTS: float32
    [T*k, N]; ROM_PROJ_CONV_GATE_SLOTS (with q1, s1): float32 [2, T*k, N]."""
    if stream is None and _fast is not None and _fast_done(
            _fast.expert_proj_w4(proj, x, q0, s0, q1, s1, N, k, topk_idx, topk_w, out),
            "rom_expert_proj_w4"):
        return
    T, K = x.shape
    E, nt, kb = q0.shape[:3]
    dev = _device(x, "x")
    if nt != -(-N // 16) or kb != -(-K // 128):
        raise RomError(f"q0 {list(q0.shape)} does not hold {N} x {K} weights")
    groups = s0.shape[-1]
    if groups not in (1, 2, 4):
        raise RomError("s0 must hold 1, 2 or 4 scales per row and tile")
    gate = proj == ROM_PROJ_CONV_GATE_SLOTS
    if gate != (q1 is not None) or gate != (s1 is not None):
        raise RomError("q1 and s1 go with ROM_PROJ_CONV_GATE_SLOTS, and only with it")
    if gate:
        po = _t(out, "out", _F32, (2, T * k, N), dev)
    elif k == 1 and proj != ROM_PROJ_SLOTS:
        po = _t(out, "out", _BF16, (T, N), dev)
    else:
        po = _t(out, "out", _F32, (T * k, N), dev)
    qs, ss = (E, nt, kb, 2, 8, 4, 16), (E, nt, kb, 16, groups)
    _call("rom_expert_proj_w4", dev, stream, proj, _t(x, "x", _BF16, (T, K), dev), T, K,
          _t(q0, "q0", torch.uint8, qs, dev), _t(s0, "s0", _BF16, ss, dev),
          _t(q1, "q1", torch.uint8, qs, dev) if gate else None,
          _t(s1, "s1", _BF16, ss, dev) if gate else None, N, E, k, 128 // groups,
          _t(topk_idx, "topk_idx", _I32, (T, k), dev),
          None if topk_w is None else _t(topk_w, "topk_w", _F32, (T, k), dev), po)


# ------------------------------------------------------------------ block helpers


def expert_weight_layout(w_pages: torch.Tensor) -> torch.Tensor:
    """[E, K, N] (the pages' x W notation) -> the library's [E, N, K] layout."""
    return w_pages.transpose(1, 2).contiguous()


class RoutingBuffers:
    """Device buffers of one routing + dispatch pass (allocated by torch)."""

    def __init__(self, T, Dm, E, k, dtype, device):
        R = T * k
        self.T, self.Dm, self.E, self.k = T, Dm, E, k
        self.topk_idx = torch.empty((T, k), dtype=torch.int32, device=device)
        self.topk_w = torch.empty((T, k), dtype=torch.float32, device=device)
        self.counts = torch.empty((E,), dtype=torch.int32, device=device)
        nws = max(1, rom_workspace_size(T, E) // 4)
        self.ws = torch.empty((nws,), dtype=torch.int32, device=device)
        self.offsets = torch.empty((E + 1,), dtype=torch.int32, device=device)
        self.sorted_slot = torch.empty((max(R, 1),), dtype=torch.int32, device=device)
        self.slot_pos = torch.empty((max(R, 1),), dtype=torch.int32, device=device)
        self.x_sorted = torch.empty((max(R, 1), Dm), dtype=dtype, device=device)


def route_and_dispatch(x, w_r, bias, E, k, renorm, bufs=None, stream=None):
    T, Dm = x.shape
    if bufs is None:
        bufs = RoutingBuffers(T, Dm, E, k, x.dtype, x.device)
    rom_route(x, w_r, bias, k, renorm, bufs.topk_idx, bufs.topk_w, bufs.counts, bufs.ws, stream)
    rom_dispatch(x, E, k, bufs.topk_idx, bufs.ws, bufs.offsets, bufs.sorted_slot, bufs.slot_pos,
                 bufs.x_sorted, stream)
    return bufs


# ------------------------------------------------------------------ dense core


class CoreParams:
    """The dense core's parameters on the device in the library's layout
    (from float32 arrays in the pages' x W notation: conv_w [De, K],
    conv_b [De], w_x [De, R + 2N], w_dt [R, De], b_dt [De], a_log [De, N],
    d [De]; w_x and w_dt must hold bf16 values). With w_x [E, De, R + 2N]
    and w_dt [E, R, De] the x and dt projections are expertized
    (``self.E`` matrices, routed with the block's selection)."""

    def __init__(self, p, device="cuda"):
        import numpy as np
        De, K = p["conv_w"].shape
        wx_p = np.asarray(p["w_x"], np.float32)
        wdt_p = np.asarray(p["w_dt"], np.float32)
        self.routed = wx_p.ndim == 3
        if not self.routed:
            wx_p, wdt_p = wx_p[None], wdt_p[None]
        self.E = wx_p.shape[0]
        self.R = wdt_p.shape[1]
        self.De = De
        self.N = p["a_log"].shape[1]
        self.K = K
        self.Np = -(-(self.R + 2 * self.N) // 128) * 128

        def f32(a):
            return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(device)
        self.conv_w, self.conv_b = f32(p["conv_w"]), f32(p["conv_b"])
        self.b_dt, self.a_log, self.d = f32(p["b_dt"]), f32(p["a_log"]), f32(p["d"])
        wx = torch.zeros((self.E, self.Np, De), dtype=torch.float32)
        wx[:, :self.R + 2 * self.N] = torch.from_numpy(np.ascontiguousarray(wx_p)).transpose(1, 2)
        self.w_x = wx.to(torch.bfloat16).to(device).contiguous()  # exact: bf16 values
        self.w_dt = torch.from_numpy(np.ascontiguousarray(wdt_p)).transpose(1, 2).contiguous() \
            .to(torch.bfloat16).to(device)


def rom_ssm_core_workspace_size(T, De, seq_len, R, N, Np):
    return int(load_library().rom_ssm_core_workspace_size(T, De, seq_len, R, N, Np))


def rom_ssm_core(h, seq_len, core, y, ws, stream=None, routing=None):
    """Y = core(H) (h, y: float32 [T, De], may be the same tensor). An
    expertized core takes the block's RoutingBuffers as ``routing``."""
    T, De = h.shape
    common = (_ptr(h), T, De, seq_len, _ptr(core.conv_w), _ptr(core.conv_b), core.K,
              _ptr(core.w_x), core.R, core.N, core.Np, _ptr(core.w_dt), _ptr(core.b_dt),
              _ptr(core.a_log), _ptr(core.d))
    tail = (_ptr(y), _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(),
            _stream(stream))
    if core.routed:
        _check(load_library().rom_ssm_core_routed(
            *common, core.E, routing.k, _ptr(routing.offsets), _ptr(routing.sorted_slot), *tail),
            "rom_ssm_core_routed")
    else:
        _check(load_library().rom_ssm_core(*common, *tail), "rom_ssm_core")


def core_workspace(T, De, seq_len, core, device, k=1):
    if core.routed:
        n = int(load_library().rom_ssm_core_routed_workspace_size(T, De, seq_len, core.R, core.N,
                                                                  core.Np, core.E, k))
    else:
        n = rom_ssm_core_workspace_size(T, De, seq_len, core.R, core.N, core.Np)
    return torch.empty((max(n, 256),), dtype=torch.uint8, device=device)


class BlockBuffers:
    """Intermediate and output buffers of one RoM block forward."""

    def __init__(self, T, Dm, De, E, k, dtype, device, core=None, seq_len=None, keep_uz=False):
        R = T * k
        self.routing = RoutingBuffers(T, Dm, E, k, dtype, device)
        self.h_sorted = torch.empty((max(R, 1), De), dtype=dtype, device=device)
        self.uz = (torch.empty((2, R, De), dtype=torch.float32, device=device)
                   if (k > 1 or core is not None or keep_uz) else None)
        self.core_ws = (core_workspace(T, De, seq_len or T, core, device, k)
                        if core is not None else None)
        self.hsum = (torch.empty((T, De), dtype=torch.float32, device=device)
                     if (core is not None and k > 1) else None)
        self.o_slots = (torch.empty((R, Dm), dtype=torch.float32, device=device)
                        if k > 1 else None)
        self.out = torch.empty((T, Dm), dtype=dtype, device=device)


def block_forward(x, w_r, bias, w_conv, w_gate, w_out, k, renorm=False, bufs=None, stream=None,
                  core=None, seq_len=None, keep_uz=False):
    """RoM block forward: route, dispatch, Conv+Gate, (gate combine), Out, (sum).

    x [T, Dm] (bf16 or float32), w_r [Dm, E] float32, bias [E] float32 or None,
    w_conv, w_gate [E, De, Dm] and w_out [E, Dm, De] in the library layout.
    ``core`` (CoreParams): the dense core runs between the projections, Y =
    core(H), over sequences of ``seq_len`` tokens (all T if None); without it
    Y = H. ``keep_uz`` (top-1): keep the float32 u and z of every token for a
    backward (the Conv+Gate projection then writes them and the gate combine
    forms h, instead of the fused u * SiLU(z) epilogue).
    Returns the BlockBuffers holding O (``.out``) and the intermediates.
    """
    T, Dm = x.shape
    E, De, _ = w_conv.shape
    if bufs is None:
        bufs = BlockBuffers(T, Dm, De, E, k, x.dtype, x.device, core, seq_len,
                            keep_uz=keep_uz)
    rb = route_and_dispatch(x, w_r, bias, E, k, renorm, bufs.routing, stream)
    R = T * k
    xs = rb.x_sorted[:R]
    if core is not None:
        # u and z per slot (float32); H in token order (the sum over the
        # slots for k > 1); Y = core(H) written just before the z rows, so
        # that [Y; z] feed the gate combine (Y per token, z per slot).
        rom_expert_proj(ROM_PROJ_CONV_GATE_SLOTS, xs, w_conv, w_gate, E, k, rb.offsets,
                        rb.sorted_slot, rb.topk_w, bufs.uz, stream)
        flat = bufs.uz.view(2 * R, De)
        y_rows = flat[R - T:R]
        if k > 1:
            rom_combine(ROM_COMBINE_SUM, ROM_F32, bufs.uz[0], T, k, De, None, bufs.hsum, stream)
            rom_ssm_core(bufs.hsum, seq_len or T, core, y_rows, bufs.core_ws, stream, rb)
        else:
            rom_ssm_core(flat[:T], seq_len or T, core, y_rows, bufs.core_ws, stream, rb)
        rom_combine(ROM_COMBINE_GATE_DENSE, _dtype_code(x), flat[R - T:], T, k, De, rb.slot_pos,
                    bufs.h_sorted, stream)
        if k == 1:
            rom_expert_proj(ROM_PROJ_OUT, bufs.h_sorted[:R], w_out, None, E, k, rb.offsets,
                            rb.sorted_slot, rb.topk_w, bufs.out, stream)
        else:
            rom_expert_proj(ROM_PROJ_OUT, bufs.h_sorted[:R], w_out, None, E, k, rb.offsets,
                            rb.sorted_slot, rb.topk_w, bufs.o_slots, stream)
            rom_combine(ROM_COMBINE_SUM, _dtype_code(x), bufs.o_slots, T, k, Dm, None, bufs.out,
                        stream)
        return bufs
    if k == 1 and keep_uz:
        if bufs.uz is None:
            raise RomError("keep_uz needs BlockBuffers made with keep_uz=True")
        rom_expert_proj(ROM_PROJ_CONV_GATE_SLOTS, xs, w_conv, w_gate, E, k, rb.offsets,
                        rb.sorted_slot, rb.topk_w, bufs.uz, stream)
        rom_combine(ROM_COMBINE_GATE, _dtype_code(x), bufs.uz, T, k, De, rb.slot_pos,
                    bufs.h_sorted, stream)
        rom_expert_proj(ROM_PROJ_OUT, bufs.h_sorted[:R], w_out, None, E, k, rb.offsets,
                        rb.sorted_slot, rb.topk_w, bufs.out, stream)
    elif k == 1:
        rom_expert_proj(ROM_PROJ_CONV_GATE, xs, w_conv, w_gate, E, k, rb.offsets, rb.sorted_slot,
                        rb.topk_w, bufs.h_sorted, stream)
        rom_expert_proj(ROM_PROJ_OUT, bufs.h_sorted[:R], w_out, None, E, k, rb.offsets,
                        rb.sorted_slot, rb.topk_w, bufs.out, stream)
    else:
        rom_expert_proj(ROM_PROJ_CONV_GATE, xs, w_conv, w_gate, E, k, rb.offsets, rb.sorted_slot,
                        rb.topk_w, bufs.uz, stream)
        rom_combine(ROM_COMBINE_GATE, _dtype_code(x), bufs.uz, T, k, De, rb.slot_pos,
                    bufs.h_sorted, stream)
        rom_expert_proj(ROM_PROJ_OUT, bufs.h_sorted[:R], w_out, None, E, k, rb.offsets,
                        rb.sorted_slot, rb.topk_w, bufs.o_slots, stream)
        rom_combine(ROM_COMBINE_SUM, _dtype_code(x), bufs.o_slots, T, k, Dm, None, bufs.out,
                    stream)
    return bufs


def inproj_forward(x, w_r, w, k=1, renorm=False, bias=None, bufs=None, out=None, slots=None,
                   stream=None, dense_small=True, w_tiled=None, w_q4=None):
    """Swimba routed in-projection: s_t = sum_j r_{t,j} x_t W_{S_j} (W as [E, N, Dm]).

    A bf16 batch of at most DENSE_SMALL_MAX_TOKENS tokens (a decode step)
    takes the projection without a dispatch (rom_expert_proj_dense) unless
    ``dense_small`` is False; the router then forms neither the per-expert
    counts nor the per-chunk histograms (``bufs.counts`` is left as it was),
    which only a dispatch needs. ``w_tiled`` (pack_expert_weights(w)), when
    given, is what that path reads instead of ``w``. ``w_q4`` (W4Weights):
    the projection runs on the 4-bit weights instead, 64 tokens at a time for
    any T, and ``w`` may be None."""
    T, Dm = x.shape
    R = T * k
    if w_q4 is not None:
        return _inproj_forward_w4(x, w_r, w_q4, k, renorm, bias, bufs, out, slots, stream)
    E, N, _ = w.shape
    if out is None:
        out = torch.empty((T, N), dtype=x.dtype, device=x.device)
    if dense_small and x.dtype == torch.bfloat16 and 0 < T <= DENSE_SMALL_MAX_TOKENS:
        if bufs is None:
            bufs = RoutingBuffers(T, Dm, E, k, x.dtype, x.device)
        rom_route(x, w_r, bias, k, renorm, bufs.topk_idx, bufs.topk_w, None, None, stream)
        wd = w if w_tiled is None else w_tiled
        tiled = w_tiled is not None
        if k == 1:
            rom_expert_proj_dense(ROM_PROJ_INPROJ, x, wd, E, k, bufs.topk_idx, bufs.topk_w, out,
                                  stream, tiled)
        else:
            if slots is None:
                slots = torch.empty((R, N), dtype=torch.float32, device=x.device)
            rom_expert_proj_dense(ROM_PROJ_INPROJ, x, wd, E, k, bufs.topk_idx, bufs.topk_w, slots,
                                  stream, tiled)
            rom_combine(ROM_COMBINE_SUM, _dtype_code(x), slots, T, k, N, None, out, stream)
        return out, bufs
    rb = route_and_dispatch(x, w_r, bias, E, k, renorm, bufs, stream)
    if k == 1:
        rom_expert_proj(ROM_PROJ_INPROJ, rb.x_sorted[:R], w, None, E, k, rb.offsets,
                        rb.sorted_slot, rb.topk_w, out, stream)
    else:
        if slots is None:
            slots = torch.empty((R, N), dtype=torch.float32, device=x.device)
        rom_expert_proj(ROM_PROJ_INPROJ, rb.x_sorted[:R], w, None, E, k, rb.offsets,
                        rb.sorted_slot, rb.topk_w, slots, stream)
        rom_combine(ROM_COMBINE_SUM, _dtype_code(x), slots, T, k, N, None, out, stream)
    return out, rb


def _inproj_forward_w4(x, w_r, w, k, renorm, bias, bufs, out, slots, stream):
    T, Dm = x.shape
    dev = _device(x, "x")
    _t(x, "x", _BF16, (T, w.K), dev)
    _t(w_r, "w_r", _F32, (Dm, w.E), dev)
    if bias is not None:
        _t(bias, "bias", _F32, (w.E,), dev)
    with _scope(x, stream):
        if bufs is None:
            bufs = RoutingBuffers(T, Dm, w.E, k, x.dtype, x.device)
        else:
            _given(bufs, dev, topk_idx=(_I32, (T, k)), topk_w=(_F32, (T, k)))
        if out is None:
            out = torch.empty((T, w.N), dtype=x.dtype, device=x.device)
        else:
            _t(out, "out", _BF16, (T, w.N), dev)
        if k > 1 and slots is None:
            slots = torch.empty((T * k, w.N), dtype=torch.float32, device=x.device)
        rom_route(x, w_r, bias, k, renorm, bufs.topk_idx, bufs.topk_w, None, None, stream)
        _w4_tokens(ROM_PROJ_INPROJ, x, w, None, k, bufs.topk_idx, bufs.topk_w,
                   out if k == 1 else slots, stream)
        if k > 1:
            rom_combine(ROM_COMBINE_SUM, _dtype_code(x), slots, T, k, w.N, None, out, stream)
    return out, bufs


# ------------------------------------------------------------------ norm, 8-bit and 4-bit blocks


def _scope(t, stream):
    """Runs the library on the device of ``t`` and on ``stream`` (None: that
    device's current one). Buffers that the functions below make belong to that
    stream, so that their memory is never still in use on another one."""
    if stream is not None and stream.device != t.device:
        raise RomError(f"the stream is one of {stream.device}, the call's first tensor on "
                       f"{t.device}")
    return torch.cuda.device(t.device) if stream is None else torch.cuda.stream(stream)


def _given(bufs, dev, **tensors):
    """Refuses buffers of another call's sizes: those that rom_route and rom_combine
    write, which take them as they come (name=(type, shape))."""
    for name, (dtype, shape) in tensors.items():
        t = getattr(bufs, name)
        if t is None:
            raise RomError(f"the buffers hold no {name}")
        _t(t, name, dtype, shape, dev)


def quant_rows(x, stream=None):
    """(codes e4m3 [rows, K], scales float32 [rows]) of x [rows, K]: 8-bit rows
    with code * scale standing for the value."""
    with _scope(x, stream):
        q = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device)
        scale = torch.empty(x.shape[:1], dtype=torch.float32, device=x.device)
        rom_quant_rows(x, q, scale, stream)
    return q, scale


class Q8Weights:
    """Expert weights [E, N, K] in 8 bits: ``q`` e4m3 and ``scale`` float32
    [E, N], one per output feature."""

    def __init__(self, q, scale):
        self.q, self.scale = q, scale
        self.E, self.N, self.K = q.shape

    @classmethod
    def quantize(cls, w, stream=None):
        """From weights [E, N, K] in bf16 or float32 (the library layout)."""
        E, N, K = w.shape
        q, scale = quant_rows(w.view(E * N, K), stream)
        return cls(q.view(E, N, K), scale.view(E, N))

    def dequantize(self):
        """The float32 values [E, N, K] that the codes stand for."""
        return self.q.float() * self.scale.unsqueeze(-1)


class W4Weights:
    """Expert weights [E, N, K] in 4 bits with a bf16 scale per ``group``
    columns, in the tiled storage of include/rom.h (``q`` and ``s``)."""

    def __init__(self, q, s, N, K):
        self.q, self.s, self.N, self.K = q, s, N, K
        self.E = q.shape[0]
        self.group = 128 // s.shape[-1]

    @classmethod
    def quantize(cls, w, group=128, stream=None):
        """From weights [E, N, K] in bf16 or float32 (the library layout)."""
        E, N, K = w.shape
        if group not in (32, 64, 128):
            raise RomError(f"group must be 32, 64 or 128, got {group}")
        nt, kb = -(-N // 16), -(-K // 128)
        with _scope(w, stream):
            q = torch.empty((E, nt, kb, 2, 8, 4, 16), dtype=torch.uint8, device=w.device)
            s = torch.empty((E, nt, kb, 16, 128 // group), dtype=torch.bfloat16, device=w.device)
            rom_quant_expert_weights_w4(w, group, q, s, stream)
        return cls(q, s, N, K)

    def dequantize(self):
        """The float32 values [E, N, K] that the codes stand for (plain torch
        operations: for checks and export, not for a hot path)."""
        E, nt, kb = self.q.shape[:3]
        v = torch.stack((self.q & 15, self.q >> 4), -1).float() - 8.0
        # .., half, 8 rows, lane, word, then the three bits of a nibble's place
        v = v.view(E, nt, kb, 2, 8, 4, 4, 2, 2, 2).permute(0, 1, 3, 4, 2, 6, 8, 5, 9, 7)
        s = self.s.float().permute(0, 1, 3, 2, 4).reshape(E, nt * 16, kb, 128 // self.group, 1)
        v = v.reshape(E, nt * 16, kb, 128 // self.group, self.group) * s
        return v.reshape(E, nt * 16, kb * 128)[:, :self.N, :self.K].contiguous()


# Tokens of one rom_expert_proj_w4 call.
W4_MAX_TOKENS = 64


def _w4_tokens(proj, x, w0, w1, k, topk_idx, topk_w, out, stream):
    """rom_expert_proj_w4 for any number of tokens, 64 at a time. ``out`` holds
    the rows of all tokens (or slots); two matrices write out[0] and out[1]."""
    T = x.shape[0]
    for a in range(0, T, W4_MAX_TOKENS):
        b = min(T, a + W4_MAX_TOKENS)
        idx, r = topk_idx[a:b], topk_w[a:b]
        if proj == ROM_PROJ_CONV_GATE_SLOTS and T > W4_MAX_TOKENS:
            # u and z of a part of the tokens are not contiguous together
            for w, o in ((w0, out[0]), (w1, out[1])):
                rom_expert_proj_w4(ROM_PROJ_SLOTS, x[a:b], w.q, w.s, None, None, w.N, k, idx, None,
                                   o[a * k:b * k], stream)
        elif proj == ROM_PROJ_CONV_GATE_SLOTS:
            rom_expert_proj_w4(proj, x, w0.q, w0.s, w1.q, w1.s, w0.N, k, idx, None, out, stream)
        else:
            rows = out[a * k:b * k]
            rom_expert_proj_w4(proj, x[a:b], w0.q, w0.s, None, None, w0.N, k, idx, r, rows, stream)


class NormBuffers:
    """Outputs of the residual norm: ``residual`` (the new residual stream),
    ``y`` (the block's input), ``rstd``, and with ``q8`` the 8-bit rows ``y8``
    and their scales ``y_scale``."""

    def __init__(self, T, D, dtype, residual_dtype, device, q8=False):
        self.residual = torch.empty((T, D), dtype=residual_dtype, device=device)
        self.y = torch.empty((T, D), dtype=dtype, device=device)
        self.rstd = torch.empty((T,), dtype=torch.float32, device=device)
        self.y8 = torch.empty((T, D), dtype=torch.float8_e4m3fn, device=device) if q8 else None
        self.y_scale = torch.empty((T,), dtype=torch.float32, device=device) if q8 else None


def add_rmsnorm(x, residual, weight, eps=1e-5, q8=False, residual_dtype=torch.float32, bufs=None,
                stream=None):
    """Residual addition and norm in front of a block (rom_add_rmsnorm). ``x``
    [T, Dm] is the block output before it (or the embeddings, with ``residual``
    None: the residual stream then starts in ``residual_dtype``). Returns
    NormBuffers."""
    T, D = x.shape
    if bufs is None:
        rt = residual_dtype if residual is None else residual.dtype
        with _scope(x, stream):
            bufs = NormBuffers(T, D, x.dtype, rt, x.device, q8)
    rom_add_rmsnorm(x, residual, weight, eps, bufs.residual, bufs.y, bufs.y8, bufs.y_scale,
                    bufs.rstd, stream)
    return bufs


class NormGrads:
    """Gradients of the residual norm: ``dx`` (also the residual's, in the
    activations' type), ``dresidual`` (the same values in the stream's type) and
    ``dw`` float32, with the call's workspace."""

    def __init__(self, T, D, dtype, residual_dtype, device):
        self.dx = torch.empty((T, D), dtype=dtype, device=device)
        self.dresidual = (self.dx if residual_dtype == dtype else
                          torch.empty((T, D), dtype=residual_dtype, device=device))
        self.dw = torch.empty((D,), dtype=torch.float32, device=device)
        n = max(16, rom_add_rmsnorm_bwd_workspace_size(T, D))
        self.ws = torch.empty((n,), dtype=torch.uint8, device=device)


def add_rmsnorm_backward(dy, norm, weight, dresidual=None, bufs=None, stream=None):
    """Backward of add_rmsnorm (``norm``: its NormBuffers): dy [T, Dm] is the
    gradient of y, ``dresidual`` that of the new residual stream from the layers
    after it (or None). Returns NormGrads."""
    T, D = dy.shape
    if bufs is None:
        with _scope(dy, stream):
            bufs = NormGrads(T, D, dy.dtype, norm.residual.dtype, dy.device)
    rom_add_rmsnorm_bwd(dy, dresidual, norm.residual, weight, norm.rstd, bufs.dx,
                        None if bufs.dresidual is bufs.dx else bufs.dresidual, bufs.dw, bufs.ws,
                        stream)
    return bufs


class Q8BlockBuffers:
    """Buffers of one 8-bit block forward; ``routing`` is a RoutingBuffers whose
    x_sorted holds e4m3 rows, with their scales in ``x_scale_sorted``."""

    def __init__(self, T, Dm, De, E, k, device):
        R, e4, f32, bf = T * k, torch.float8_e4m3fn, torch.float32, torch.bfloat16
        n = max(R, 1)
        self.x8 = torch.empty((T, Dm), dtype=e4, device=device)
        self.x_scale = torch.empty((T,), dtype=f32, device=device)
        self.routing = RoutingBuffers(T, Dm, E, k, e4, device)
        self.x_scale_sorted = torch.empty((n,), dtype=f32, device=device)
        self.uz = torch.empty((2, R, De), dtype=f32, device=device) if k > 1 else None
        self.h_sorted = torch.empty((R, De), dtype=bf, device=device)
        self.h8 = torch.empty((R, De), dtype=e4, device=device)
        self.h_scale = torch.empty((R,), dtype=f32, device=device)
        self.o_slots = torch.empty((R, Dm), dtype=f32, device=device) if k > 1 else None
        self.out = torch.empty((T, Dm), dtype=bf, device=device)


def block_forward_q8(x, w_r, bias, w_conv, w_gate, w_out, k, renorm=False, x8=None, x_scale=None,
                     bufs=None, stream=None):
    """RoM block forward with the expert projections in 8 bits (Q8Weights).

    x [T, Dm] bf16 is what the router reads; the experts read its 8-bit rows
    ``x8``, ``x_scale`` (add_rmsnorm(..., q8=True) writes them beside x), made
    here when not given. The gated rows h are rounded to bf16 and then to
    8-bit rows for the Out projection. Returns the Q8BlockBuffers (O in
    ``.out``)."""
    T, Dm = x.shape
    E, De = w_conv.E, w_conv.N
    dev = _device(x, "x")
    _t(x, "x", _BF16, (T, w_conv.K), dev)
    _t(w_r, "w_r", _F32, (Dm, E), dev)
    if bias is not None:
        _t(bias, "bias", _F32, (E,), dev)
    if (x8 is None) != (x_scale is None):
        raise RomError("x8 and x_scale come together")
    if w_gate.q.shape != w_conv.q.shape or w_out.q.shape != (E, Dm, De):
        raise RomError("the 8-bit weights' sizes do not fit together")
    if Dm % 128 or De % 128:
        raise RomError(f"d_model and d_inner must be multiples of 128, got {Dm} and {De}")
    with _scope(x, stream):
        if bufs is None:
            bufs = Q8BlockBuffers(T, Dm, De, E, k, x.device)
        else:
            _given(bufs.routing, dev, topk_idx=(_I32, (T, k)), topk_w=(_F32, (T, k)),
                   counts=(_I32, (E,)))
            _ws(bufs.routing.ws, dev)  # (its size: rom_route)
            _given(bufs, dev, h_sorted=(_BF16, (T * k, De)), out=(_BF16, (T, Dm)))
        if x8 is None:
            x8, x_scale = bufs.x8, bufs.x_scale
            rom_quant_rows(x, x8, x_scale, stream)
        rb = bufs.routing
        R = T * k
        rom_route(x, w_r, bias, k, renorm, rb.topk_idx, rb.topk_w, rb.counts, rb.ws, stream)
        rom_dispatch_q8(x8, x_scale, E, k, rb.topk_idx, rb.ws, rb.offsets, rb.sorted_slot,
                        rb.slot_pos, rb.x_sorted, bufs.x_scale_sorted, stream)
        rom_expert_proj_q8(ROM_PROJ_CONV_GATE, rb.x_sorted[:R], bufs.x_scale_sorted[:R], w_conv.q,
                           w_conv.scale, w_gate.q, w_gate.scale, k, rb.offsets, rb.sorted_slot,
                           rb.topk_w, bufs.h_sorted if k == 1 else bufs.uz, stream)
        if k > 1:
            rom_combine(ROM_COMBINE_GATE, ROM_BF16, bufs.uz, T, k, De, rb.slot_pos, bufs.h_sorted,
                        stream)
        rom_quant_rows(bufs.h_sorted, bufs.h8, bufs.h_scale, stream)
        rom_expert_proj_q8(ROM_PROJ_OUT, bufs.h8, bufs.h_scale, w_out.q, w_out.scale, None, None, k,
                           rb.offsets, rb.sorted_slot, rb.topk_w,
                           bufs.out if k == 1 else bufs.o_slots, stream)
        if k > 1:
            rom_combine(ROM_COMBINE_SUM, ROM_BF16, bufs.o_slots, T, k, Dm, None, bufs.out, stream)
    return bufs


class W4BlockBuffers:
    """Buffers of one block forward on 4-bit weights."""

    def __init__(self, T, Dm, De, k, device):
        R, f32, bf = T * k, torch.float32, torch.bfloat16
        self.topk_idx = torch.empty((T, k), dtype=torch.int32, device=device)
        self.topk_w = torch.empty((T, k), dtype=f32, device=device)
        self.uz = torch.empty((2, R, De), dtype=f32, device=device)
        self.h = torch.empty((T, De), dtype=bf, device=device)
        self.o_slots = torch.empty((R, Dm), dtype=f32, device=device) if k > 1 else None
        self.out = torch.empty((T, Dm), dtype=bf, device=device)


def block_forward_w4(x, w_r, bias, w_conv, w_gate, w_out, k, renorm=False, bufs=None, stream=None):
    """RoM block forward of a decode batch on 4-bit expert weights (W4Weights):
    route, Conv+Gate, gate combine, Out, (sum), all in token order without a
    dispatch. Any T, 64 tokens at a time; meant for few. x [T, Dm] bf16.
    Returns the W4BlockBuffers (O in ``.out``)."""
    T, Dm = x.shape
    dev = _device(x, "x")
    _t(x, "x", _BF16, (T, w_conv.K), dev)
    _t(w_r, "w_r", _F32, (Dm, w_conv.E), dev)
    if bias is not None:
        _t(bias, "bias", _F32, (w_conv.E,), dev)
    if w_out.K != w_conv.N or w_out.N != Dm or w_gate.q.shape != w_conv.q.shape:
        raise RomError("the 4-bit weights' sizes do not fit together")
    De = w_conv.N
    with _scope(x, stream):
        if bufs is None:
            bufs = W4BlockBuffers(T, Dm, De, k, x.device)
        else:
            _given(bufs, dev, topk_idx=(_I32, (T, k)), topk_w=(_F32, (T, k)),
                   h=(_BF16, (T, De)), out=(_BF16, (T, Dm)))
        rom_route(x, w_r, bias, k, renorm, bufs.topk_idx, bufs.topk_w, None, None, stream)
        _w4_tokens(ROM_PROJ_CONV_GATE_SLOTS, x, w_conv, w_gate, k, bufs.topk_idx, bufs.topk_w,
                   bufs.uz, stream)
        rom_combine(ROM_COMBINE_GATE, ROM_BF16, bufs.uz, T, k, De, None, bufs.h, stream)
        _w4_tokens(ROM_PROJ_OUT, bufs.h, w_out, None, k, bufs.topk_idx, bufs.topk_w,
                   bufs.out if k == 1 else bufs.o_slots, stream)
        if k > 1:
            rom_combine(ROM_COMBINE_SUM, ROM_BF16, bufs.o_slots, T, k, Dm, None, bufs.out, stream)
    return bufs


class ResidualBlock:
    """One pre-norm block: ``norm`` (NormBuffers) and ``block`` (the block's
    buffers); ``out`` is the block's output, ``residual`` the residual stream
    that the next block's norm adds it to. ``renorm``: as the block ran."""

    def __init__(self, norm, block, renorm):
        self.norm, self.block, self.renorm = norm, block, renorm
        self.out, self.residual = block.out, norm.residual


def residual_block_forward(x, residual, norm_w, w_r, bias, w_conv, w_gate, w_out, k, renorm=False,
                           eps=1e-5, residual_dtype=torch.float32, norm_bufs=None, bufs=None,
                           stream=None, keep_uz=False):
    """Residual addition, norm and RoM block: block(norm(x + residual)).

    x [T, Dm]: the previous block's output; residual [T, Dm] or None (first
    block). The weights' type chooses the block: tensors (block_forward, bf16
    or float32), Q8Weights (block_forward_q8, the norm writing the 8-bit rows)
    or W4Weights (block_forward_w4). Returns a ResidualBlock."""
    q8 = isinstance(w_conv, Q8Weights)
    norm = add_rmsnorm(x, residual, norm_w, eps, q8, residual_dtype, norm_bufs, stream)
    args = (norm.y, w_r, bias, w_conv, w_gate, w_out, k, renorm)
    if q8:
        block = block_forward_q8(*args, x8=norm.y8, x_scale=norm.y_scale, bufs=bufs, stream=stream)
    elif isinstance(w_conv, W4Weights):
        block = block_forward_w4(*args, bufs=bufs, stream=stream)
    else:
        with _scope(x, stream):
            block = block_forward(*args, bufs=bufs, stream=stream, keep_uz=keep_uz)
    return ResidualBlock(norm, block, renorm)


def residual_block_backward(fwd, dout, norm_w, w_r, w_conv, w_gate, w_out, renorm=None, bias=None,
                            dresidual=None, bufs=None, norm_bufs=None, stream=None,
                            grad_sync=None):
    """Backward of residual_block_forward on bf16 weights: dout [T, Dm] is the
    gradient of the block's output, ``dresidual`` that of the residual stream
    from the layers after it (or None). Returns (BackwardBuffers, NormGrads):
    the expert and router gradients, and dx / dresidual of the block's inputs
    with the norm weight's dw. ``renorm``: None (as the forward ran) or that same
    value. With ``grad_sync`` the norm weight's gradient is summed over the ranks
    too."""
    if not isinstance(fwd.block, BlockBuffers):
        raise RomError("the blocks on 8-bit and 4-bit weights have no backward")
    if renorm is None:
        renorm = fwd.renorm
    elif bool(renorm) != bool(fwd.renorm):
        raise RomError(f"the forward ran with renorm={fwd.renorm}")
    with _scope(dout, stream):
        bwd = block_backward(fwd.block, dout, w_r, w_conv, w_gate, w_out, renorm, bufs, stream,
                             x=fwd.norm.y, bias=bias, grad_sync=grad_sync)
        grads = add_rmsnorm_backward(bwd.dx, fwd.norm, norm_w, dresidual, norm_bufs, stream)
        if grad_sync is not None:
            grad_sync.start(grads.dw)
            grad_sync.finish()
    return bwd, grads


# ------------------------------------------------------------------ projection variants

PROJECTIONS = ("conv", "gate", "out")


class VariantBuffers:
    """Buffers of one forward of a projection variant (allocated by torch)."""

    def __init__(self, T, Dm, De, k, dtype, device):
        R = T * k
        self.routings = {}  # id(router weight) -> RoutingBuffers, made on first use
        self.uz = torch.empty((2 * R, De), dtype=torch.float32, device=device)
        self.h = torch.empty((R, De), dtype=dtype, device=device)
        self.o_slots = torch.empty((R, Dm), dtype=torch.float32, device=device)
        self.out = torch.empty((T, Dm), dtype=dtype, device=device)


def variant_block_forward(x, routers, weighted, w_conv, w_gate, w_out, k, renorm=False,
                          bias=None, bufs=None, stream=None,
                          phases=("route", "project", "output")):
    """Projection block with each of Conv, Gate and Out dense or routed.

    routers: {"conv", "gate", "out"} -> router weight [Dm, E] float32, or None
    for a dense projection (its weight stack then holds one matrix). The same
    tensor passed for several projections is one shared routing decision
    (routed and dispatched once). weighted: the same keys -> True when that
    projection's expert outputs are scaled by its routing weights (Out must
    be weighted when routed). Weights in the library layout [E, N, K].

    Independently routed MoE-Mamba (RoM page, Knowl 4) passes three routers
    and weights all three; RoM (Gate, Out) (Knowl 3) passes None for Conv and
    one router for Gate and Out. Returns the VariantBuffers (O in ``.out``).

    ``phases`` runs a subset of the three steps, in order, on ``bufs`` from
    an earlier call: "route" (route and dispatch every distinct router),
    "project" (the Conv and Gate projections to float32 rows) and "output"
    (the gate combine and the Out projection).
    """
    T, Dm = x.shape
    De = w_conv.shape[1]
    R = T * k
    if routers["out"] is not None and not weighted["out"]:
        raise RomError("a routed Out projection is weighted by its routing weights")
    if routers["gate"] is None and routers["conv"] is not None and k > 1:
        raise RomError("a dense Gate projection with routed Conv needs k == 1")
    if bufs is None:
        bufs = VariantBuffers(T, Dm, De, k, x.dtype, x.device)
    wts = {"conv": w_conv, "gate": w_gate, "out": w_out}
    rbs = {}
    for n in PROJECTIONS:
        w_r = routers[n]
        if w_r is None:
            rbs[n] = None
            continue
        key = id(w_r)
        if key not in bufs.routings:
            bufs.routings[key] = RoutingBuffers(T, Dm, w_r.shape[1], k, x.dtype, x.device)
        rb = bufs.routings[key]
        # route each distinct router once
        if "route" in phases and not any(rbs.get(m) is rb for m in rbs):
            route_and_dispatch(x, w_r, bias, w_r.shape[1], k, renorm, rb, stream)
        rbs[n] = rb

    def project_slots(name, dst):
        rb = rbs[name]
        if rb is None:  # dense: one matrix over the tokens in order
            rom_expert_proj(ROM_PROJ_SLOTS, x, wts[name], None, 1, 1, None, None, None, dst,
                            stream)
        else:
            rom_expert_proj(ROM_PROJ_SLOTS, rb.x_sorted[:R], wts[name], None, wts[name].shape[0],
                            k, rb.offsets, rb.sorted_slot, rb.topk_w if weighted[name] else None,
                            dst, stream)

    conv_rows = T if rbs["conv"] is None else R
    gate_rows = T if rbs["gate"] is None else R
    if "project" in phases:
        project_slots("conv", bufs.uz[:conv_rows])
        project_slots("gate", bufs.uz[conv_rows:conv_rows + gate_rows])
    if "output" not in phases:
        return bufs
    rb_o = rbs["out"]
    dt = _dtype_code(x)
    h_pos = None if rb_o is None else rb_o.slot_pos
    h_rows = T if rb_o is None else R
    if rbs["conv"] is None and k > 1:
        rom_combine(ROM_COMBINE_GATE_DENSE, dt, bufs.uz[:T + R], T, k, De, h_pos, bufs.h, stream)
    else:
        # both Conv and Gate routed (u and z per slot), or k == 1 (a dense one
        # has one row per token, which is also its slot)
        rom_combine(ROM_COMBINE_GATE, dt, bufs.uz[:2 * R], T, k, De, h_pos, bufs.h, stream)
    if rb_o is None:
        rom_expert_proj(ROM_PROJ_SLOTS, bufs.h[:T], w_out, None, 1, 1, None, None, None,
                        bufs.o_slots[:T], stream)
        rom_combine(ROM_COMBINE_SUM, dt, bufs.o_slots[:T], T, 1, Dm, None, bufs.out, stream)
    elif k == 1:
        rom_expert_proj(ROM_PROJ_OUT, bufs.h[:h_rows], w_out, None, w_out.shape[0], k,
                        rb_o.offsets, rb_o.sorted_slot, rb_o.topk_w, bufs.out, stream)
    else:
        rom_expert_proj(ROM_PROJ_OUT, bufs.h[:h_rows], w_out, None, w_out.shape[0], k,
                        rb_o.offsets, rb_o.sorted_slot, rb_o.topk_w, bufs.o_slots, stream)
        rom_combine(ROM_COMBINE_SUM, dt, bufs.o_slots, T, k, Dm, None, bufs.out, stream)
    return bufs


# ------------------------------------------------------------------ backward


def rom_bwd_gather(dout, k, sorted_slot, topk_w, rdo_sorted, stream=None):
    T, N = dout.shape
    _check(load_library().rom_bwd_gather(_ptr(dout), T, k, N, _ptr(sorted_slot), _ptr(topk_w),
                                         _ptr(rdo_sorted), _stream(stream)), "rom_bwd_gather")


def rom_bwd_dgrad_out(rdo_sorted, w_out, E, k, offsets, sorted_slot, h_sorted, g_slots, dr_part,
                      stream=None):
    R, Dm = rdo_sorted.shape
    De = w_out.shape[2]
    _check(load_library().rom_bwd_dgrad_out(
        _ptr(rdo_sorted), R, Dm, _ptr(w_out), De, E, k, _ptr(offsets), _ptr(sorted_slot),
        _ptr(h_sorted), _ptr(g_slots), _ptr(dr_part), _stream(stream)), "rom_bwd_dgrad_out")


def rom_bwd_gate(uz, g_slots, T, k, De, slot_pos, dhz_sorted, stream=None):
    _check(load_library().rom_bwd_gate(_ptr(uz), _ptr(g_slots), T, k, De, _ptr(slot_pos),
                                       _ptr(dhz_sorted), _stream(stream)), "rom_bwd_gate")


def rom_bwd_dgrad_in(dhz_sorted, w_in, w_g, E, k, offsets, sorted_slot, dx_slots, stream=None):
    R = dhz_sorted.shape[0]
    De = dhz_sorted.shape[1] // 2
    Dm = w_in.shape[2]
    _check(load_library().rom_bwd_dgrad_in(
        _ptr(dhz_sorted), R, De, _ptr(w_in), _ptr(w_g), Dm, E, k, _ptr(offsets),
        _ptr(sorted_slot), _ptr(dx_slots), _stream(stream)), "rom_bwd_dgrad_in")


def rom_route_bwd(T, k, E, Dm, renorm, topk_idx, topk_w, dr_part, dx_slots, w_r, dlogits, dx,
                  stream=None, probs=None):
    _check(load_library().rom_route_bwd(
        T, k, E, Dm, int(renorm), _ptr(topk_idx), _ptr(topk_w), _ptr(probs), _ptr(dr_part),
        dr_part.shape[1], _ptr(dx_slots), _ptr(w_r), _ptr(dlogits), _ptr(dx), _stream(stream)),
        "rom_route_bwd")


def rom_route_probs(x, w_r, bias, probs, stream=None):
    T, Dm = x.shape
    _check(load_library().rom_route_probs(_ptr(x), _dtype_code(x), T, Dm, _ptr(w_r), _ptr(bias),
                                          w_r.shape[1], _ptr(probs), _stream(stream)),
           "rom_route_probs")


def rom_route_wgrad(x, dlogits, dw_r, dbias, stream=None):
    T, Dm = x.shape
    _check(load_library().rom_route_wgrad(_ptr(x), _dtype_code(x), T, Dm, dlogits.shape[1],
                                          _ptr(dlogits), _ptr(dw_r), _ptr(dbias),
                                          _stream(stream)), "rom_route_wgrad")


def rom_bwd_wgrad(a_sorted, b_sorted, E, offsets, m_split, out0, out1, stream=None):
    R, M = a_sorted.shape
    N = b_sorted.shape[1]
    _check(load_library().rom_bwd_wgrad(
        _ptr(a_sorted), M, _ptr(b_sorted), N, R, E, _ptr(offsets), m_split, _ptr(out0),
        _ptr(out1), _stream(stream)), "rom_bwd_wgrad")


class GradientAllReduce:
    """Data-parallel exchange of the weight gradients: every rank holds the
    gradients of its own tokens, and each tensor handed to ``start`` is summed
    over the ranks of ``group`` (torch.distributed all-reduce: NCCL over
    NVLink between GPUs, gloo between CPU processes). A transfer is started
    as soon as the kernel that produces its tensor is enqueued, so it overlaps
    the rest of the backward; ``finish`` makes the current stream wait for
    all of them. Every rank must start the same tensors in the same order.
    The token batch is split across ranks and the expert and router weights
    are replicated; the tokens themselves are never exchanged."""

    def __init__(self, group=None):
        self.group = group
        self.pending = []

    def start(self, *tensors):
        import torch.distributed as dist
        for t in tensors:
            self.pending.append(dist.all_reduce(t, op=dist.ReduceOp.SUM, group=self.group,
                                                async_op=True))

    def finish(self):
        for w in self.pending:
            w.wait()
        self.pending = []


class BackwardBuffers:
    """Device buffers of one backward pass (allocated by torch)."""

    def __init__(self, T, Dm, De, E, k, device):
        R = T * k
        bf = torch.bfloat16
        self.rdo_sorted = torch.empty((R, Dm), dtype=bf, device=device)
        self.g_slots = torch.empty((R, De), dtype=torch.float32, device=device)
        self.dr_part = torch.empty((R, De // 256), dtype=torch.float32, device=device)
        self.dhz_sorted = torch.empty((R, 2 * De), dtype=bf, device=device)
        self.dx_slots = torch.empty((R, Dm), dtype=torch.float32, device=device)
        self.dx = torch.empty((T, Dm), dtype=bf, device=device)
        self.dlogits = torch.empty((T, E), dtype=torch.float32, device=device)
        self.dw_out = torch.empty((E, Dm, De), dtype=torch.float32, device=device)
        self.dw_conv = torch.empty((E, De, Dm), dtype=torch.float32, device=device)
        self.dw_gate = torch.empty((E, De, Dm), dtype=torch.float32, device=device)
        self.dw_r = torch.empty((Dm, E), dtype=torch.float32, device=device)
        self.dbias = torch.empty((E,), dtype=torch.float32, device=device)
        self.probs = torch.empty((T, E), dtype=torch.float32, device=device)


def block_backward(fwd, dout, w_r, w_conv, w_gate, w_out, renorm=True, bufs=None, stream=None,
                   x=None, bias=None, grad_sync=None):
    """Backward of the RoM block (renormalised weights, or r = p with ``x``).

    fwd: the BlockBuffers of the forward (routing, h_sorted, u/z slot
    partials: for k == 1 the forward must have run with keep_uz=True);
    dout [T, Dm] bf16; weights in the library layout. With ``x`` (the
    forward's input) the router weight gradients dw_r [Dm, E] and dbias [E]
    are computed too; r = p (renorm=False) needs ``x`` (and the forward's
    ``bias``) for the softmax over all experts. Returns BackwardBuffers with
    dx [T, Dm] bf16, dlogits [T, E] and dw_conv / dw_gate [E, De, Dm],
    dw_out [E, Dm, De] (float32, the weights' layout).
    ``grad_sync`` (a GradientAllReduce): data-parallel training; the weight
    gradients are summed over its ranks, dW_out while the rest of the
    backward runs.
    """
    rb = fwd.routing
    T, Dm = dout.shape
    E, De, _ = w_conv.shape
    k = rb.k
    if fwd.uz is None:
        raise RomError("block_backward needs the forward's u/z slot partials "
                       "(top-k > 1, or block_forward(..., keep_uz=True))")
    if not renorm and x is None:
        raise RomError("the backward of r = p needs the forward's input x")
    R = T * k
    if bufs is None:
        bufs = BackwardBuffers(T, Dm, De, E, k, dout.device)
    rom_bwd_gather(dout, k, rb.sorted_slot, rb.topk_w, bufs.rdo_sorted, stream)
    rom_bwd_dgrad_out(bufs.rdo_sorted, w_out, E, k, rb.offsets, rb.sorted_slot,
                      fwd.h_sorted[:R], bufs.g_slots, bufs.dr_part, stream)
    if grad_sync is not None:
        # dW_out first, so that its exchange overlaps the rest of the backward
        rom_bwd_wgrad(bufs.rdo_sorted, fwd.h_sorted[:R], E, rb.offsets, Dm, bufs.dw_out, None,
                      stream)
        grad_sync.start(bufs.dw_out)
    rom_bwd_gate(fwd.uz, bufs.g_slots, T, k, De, rb.slot_pos, bufs.dhz_sorted, stream)
    rom_bwd_dgrad_in(bufs.dhz_sorted, w_conv, w_gate, E, k, rb.offsets, rb.sorted_slot,
                     bufs.dx_slots, stream)
    if not renorm:
        rom_route_probs(x, w_r, bias, bufs.probs, stream)
    rom_route_bwd(T, k, E, Dm, renorm, rb.topk_idx, rb.topk_w, bufs.dr_part, bufs.dx_slots, w_r,
                  bufs.dlogits, bufs.dx, stream, probs=None if renorm else bufs.probs)
    if x is not None:
        rom_route_wgrad(x, bufs.dlogits, bufs.dw_r, bufs.dbias, stream)
        if grad_sync is not None:
            grad_sync.start(bufs.dw_r, bufs.dbias)
    if grad_sync is None:
        rom_bwd_wgrad(bufs.rdo_sorted, fwd.h_sorted[:R], E, rb.offsets, Dm, bufs.dw_out, None,
                      stream)
    rom_bwd_wgrad(bufs.dhz_sorted, rb.x_sorted[:R], E, rb.offsets, De, bufs.dw_conv, bufs.dw_gate,
                  stream)
    if grad_sync is not None:
        grad_sync.start(bufs.dw_conv, bufs.dw_gate)
        grad_sync.finish()
    return bufs


# ------------------------------------------------------------------ host buffers, pipelined


class HostPipeline:
    """Forward of the block (or the Swimba in-projection) on HOST tensors.

    Tokens are independent, so the batch is cut into chunks (multiples of the
    128-token routing chunk) that go through three stages, each on streams of
    its own: the host-to-device copies on one stream, the kernels on two
    (a chunk of a few thousand tokens leaves the GPU room for a second one),
    the device-to-host copies on one, chained by events. The input copy of one
    chunk, the kernels of the previous ones and the output copy of an earlier
    one run at the same time, and the two copy directions overlap on the
    link. `nstreams` device buffer sets rotate over the chunks; a set takes a
    new chunk once its last chunk's output copy has completed. Each token's
    routing is the one a single call on the whole batch gives, and so is its
    output when the chunk and the batch take the same projection kernels
    (more than 1024 routed rows each); a short last chunk may take the
    swap-AB Out GEMM, whose output agrees within the forward's tolerance.
    Chunks of 2048 tokens and four buffer sets measured best for the prefill
    batch (smaller chunks cost more GEMM efficiency than the shorter first
    and last copies save). Device buffers are allocated once (torch); the
    kernels are the library's.

    With ``graph=True`` the second call with the same host buffers, weights
    and size captures the whole multi-stream sequence (copies and kernels)
    into a CUDA graph, and later such calls replay it: the host then issues
    one launch per call instead of some ten per chunk. The first call runs
    eagerly (it also initialises the library's per-device state).
    """

    def __init__(self, T, Dm, N_out, E, k, dtype, device="cuda", chunks=8, nstreams=4,
                 De=None, graph=True, min_chunk=2048):
        self.T, self.Dm, self.E, self.k = T, Dm, E, k
        self.graph = graph
        self._graphs, self._seen, self._tail = {}, set(), {}
        per = -(-T // chunks)
        # Chunks of at least min_chunk tokens (smaller ones lose more GEMM
        # efficiency and launch time than their shorter first and last copies
        # save), at most the batch.
        self.chunk = min(max(min_chunk, -(-per // 128) * 128), max(128, -(-T // 128) * 128))
        self.nbuf = nstreams
        self.s_in = torch.cuda.Stream(device=device)
        self.s_out = torch.cuda.Stream(device=device)
        self.s_comp = [torch.cuda.Stream(device=device) for _ in range(2)]
        self.x = [torch.empty((self.chunk, Dm), dtype=dtype, device=device) for _ in range(nstreams)]
        if De is not None:  # RoM block
            self.bufs = [BlockBuffers(self.chunk, Dm, De, E, k, dtype, device) for _ in range(nstreams)]
        else:  # in-projection
            self.bufs = [RoutingBuffers(self.chunk, Dm, E, k, dtype, device) for _ in range(nstreams)]
            self.out = [torch.empty((self.chunk, N_out), dtype=dtype, device=device)
                        for _ in range(nstreams)]
            self.slots = ([torch.empty((self.chunk * k, N_out), dtype=torch.float32, device=device)
                           for _ in range(nstreams)] if k > 1 else [None] * nstreams)

    def _chunks(self, T):
        return [(i, min(T, i + self.chunk)) for i in range(0, T, self.chunk)]

    def _run(self, T, body):
        """body = (copy_in, compute, copy_out), each called (j, a, b, stream)
        for every chunk [a, b) with buffer set j: one chunk runs on the
        current stream, several go through the staged streams."""
        copy_in, compute, copy_out = body
        cur = torch.cuda.current_stream()
        chunks = self._chunks(T)
        if len(chunks) == 1:
            for f in body:
                f(0, 0, T, cur)
            return
        start = torch.cuda.Event()
        start.record(cur)
        streams = [self.s_in, self.s_out] + self.s_comp
        for s in streams:
            s.wait_event(start)
        free = [None] * self.nbuf  # buffer set j: its last output copy
        for n, (a, b) in enumerate(chunks):
            j = n % self.nbuf
            with torch.cuda.stream(self.s_in):
                if free[j] is not None:
                    self.s_in.wait_event(free[j])
                copy_in(j, a, b, self.s_in)
                e_in = torch.cuda.Event()
                e_in.record(self.s_in)
            sc = self.s_comp[n % len(self.s_comp)]
            with torch.cuda.stream(sc):
                sc.wait_event(e_in)
                compute(j, a, b, sc)
                e_c = torch.cuda.Event()
                e_c.record(sc)
            with torch.cuda.stream(self.s_out):
                self.s_out.wait_event(e_c)
                copy_out(j, a, b, self.s_out)
                free[j] = torch.cuda.Event()
                free[j].record(self.s_out)
        for s in streams:
            ev = torch.cuda.Event()
            ev.record(s)
            cur.wait_event(ev)

    def _launch(self, key, T, body):
        """Eager on the first call for `key`, captured into a CUDA graph on
        the second, replayed afterwards."""
        if not self.graph:
            self._run(T, body)
            return
        g = self._graphs.get(key)
        if g is None and key in self._seen:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                self._run(T, body)
            self._graphs[key] = g
        if g is None:
            self._seen.add(key)
            self._run(T, body)
        else:
            g.replay()

    def _tail_bufs(self, n, make):
        """Buffers of a shorter last chunk, made once per size (outside any capture)."""
        if n not in self._tail:
            self._tail[n] = make(n)
        return self._tail[n]

    def block_forward(self, x_host, w_r, bias, w_conv, w_gate, w_out, out_host, renorm=False):
        """x_host [T, Dm] and out_host [T, Dm]: pinned host tensors."""
        T = x_host.shape[0]
        De = w_conv.shape[1]
        for a, b in self._chunks(T):
            if b - a != self.chunk:
                self._tail_bufs(b - a, lambda n: BlockBuffers(n, self.Dm, De, self.E, self.k,
                                                              self.x[0].dtype, self.x[0].device))

        def bufs_of(j, a, b):
            return self.bufs[j] if b - a == self.chunk else self._tail[b - a]

        def copy_in(j, a, b, s):
            self.x[j][: b - a].copy_(x_host[a:b], non_blocking=True)

        def compute(j, a, b, s):
            block_forward(self.x[j][: b - a], w_r, bias, w_conv, w_gate, w_out, self.k, renorm,
                          bufs_of(j, a, b), stream=s)

        def copy_out(j, a, b, s):
            out_host[a:b].copy_(bufs_of(j, a, b).out, non_blocking=True)

        body = (copy_in, compute, copy_out)

        key = ("block", T, x_host.data_ptr(), out_host.data_ptr(), w_r.data_ptr(),
               0 if bias is None else bias.data_ptr(), w_conv.data_ptr(), w_gate.data_ptr(),
               w_out.data_ptr(), bool(renorm))
        self._launch(key, T, body)
        return out_host

    def inproj_forward(self, x_host, w_r, w, out_host, renorm=False, bias=None, w_tiled=None):
        """x_host [T, Dm], out_host [T, N_out]: pinned host tensors."""
        T = x_host.shape[0]
        for a, b in self._chunks(T):
            if b - a != self.chunk:
                self._tail_bufs(b - a, lambda n: RoutingBuffers(n, self.Dm, self.E, self.k,
                                                                self.x[0].dtype, self.x[0].device))

        def copy_in(j, a, b, s):
            self.x[j][: b - a].copy_(x_host[a:b], non_blocking=True)

        def compute(j, a, b, s):
            bufs = self.bufs[j] if b - a == self.chunk else self._tail[b - a]
            sl = None if self.slots[j] is None else self.slots[j][: (b - a) * self.k]
            inproj_forward(self.x[j][: b - a], w_r, w, self.k, renorm, bias, bufs,
                           self.out[j][: b - a], sl, stream=s, w_tiled=w_tiled)

        def copy_out(j, a, b, s):
            out_host[a:b].copy_(self.out[j][: b - a], non_blocking=True)

        body = (copy_in, compute, copy_out)

        key = ("inproj", T, x_host.data_ptr(), out_host.data_ptr(), w_r.data_ptr(), w.data_ptr(),
               0 if bias is None else bias.data_ptr(), bool(renorm),
               0 if w_tiled is None else w_tiled.data_ptr())
        self._launch(key, T, body)
        return out_host
