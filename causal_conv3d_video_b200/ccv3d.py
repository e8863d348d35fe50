"""ctypes binding of libccv3d (include/ccv3d.h): argument marshalling only.

Every function here has the name of the C entry point it calls.  Device
buffers are passed as torch tensors (their data pointers) or as raw integer
addresses; nothing is computed in Python.  If the shared library is missing
the import of this module fails loudly: there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
# CCV3D_LIBRARY=checked loads the bounds-checked build (libccv3d_checked.so:
# the same ABI, every computed device address range-checked); the tests use it
LIB_PATH = os.path.join(_HERE, "_lib", "libccv3d_checked.so"
                        if os.environ.get("CCV3D_LIBRARY") == "checked" else "libccv3d.so")

CCV3D_BF16, CCV3D_FP32 = 0, 1
STATUS = {0: "CCV3D_OK", 1: "CCV3D_ERR_INVALID", 2: "CCV3D_ERR_UNSUPPORTED",
          3: "CCV3D_ERR_EMPTY_OUTPUT", 4: "CCV3D_ERR_ALIGNMENT", 5: "CCV3D_ERR_ALIAS",
          6: "CCV3D_ERR_CUDA", 7: "CCV3D_ERR_TIMEOUT", 8: "CCV3D_ERR_SCRATCH_LIMIT",
          9: "CCV3D_ERR_BOUNDS"}
for _code, _name in STATUS.items():
    globals()[_name] = _code
CCV3D_MAX_KT = 3

# every symbol include/ccv3d.h declares
EXPORTED = ("ccv3d_plan", "ccv3d_plan_intervals", "ccv3d_plan_path", "ccv3d_forward",
            "ccv3d_get_stats", "ccv3d_get_status", "ccv3d_destroy", "ccv3d_strerror",
            "ccv3d_plan_sizes", "ccv3d_selftest_wait_timeout", "ccv3d_forward_noalloc",
            "ccv3d_plan_kernel", "ccv3d_plan_tiling", "ccv3d_quantize_u8",
            "ccv3d_get_status_stream", "ccv3d_noalloc_get_status", "ccv3d_forward_ring",
            "ccv3d_selftest_bounds", "ccv3d_norm_forward", "ccv3d_norm_workspace",
            "ccv3d_norm_backward", "ccv3d_pointwise_workspace", "ccv3d_pointwise_forward",
            "ccv3d_pointwise_backward", "ccv3d_qcache_sizes", "ccv3d_qcache_write",
            "ccv3d_qcache_read", "ccv3d_forward_qring", "ccv3d_block_get_status")
CCV3D_NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024


class ccv3d_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "N", "Cin", "Cout", "kt", "kh", "kw", "H", "W", "T_x", "cache_len",
        "pad_t_base", "cache_keep", "stride_t", "stride_h", "stride_w", "pad_h",
        "pad_w", "dil_t", "dil_h", "dil_w", "groups", "dtype", "has_bias")]


class ccv3d_stats(ctypes.Structure):
    _fields_ = [(n, ctypes.c_uint64) for n in (
        "calls", "tc_path", "simt_path", "unsupported", "errors", "workspace_bytes",
        "plans_unsupported")]


NORM_KINDS = {"none": 0, "rms": 1, "layer": 2}
ACTS = {"none": 0, "silu": 1, "gelu": 2}
QFORMATS = {"int8": 0, "e4m3": 1, "e2m1": 2}


class ccv3d_norm_desc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_longlong), ("C", ctypes.c_int), ("pre", ctypes.c_int),
                ("post", ctypes.c_int), ("act", ctypes.c_int), ("eps", ctypes.c_float),
                ("scale", ctypes.c_float), ("gate_rows", ctypes.c_longlong),
                ("dtype", ctypes.c_int)]


class ccv3d_pointwise_desc(ctypes.Structure):
    _fields_ = [("pixels", ctypes.c_longlong), ("Cin", ctypes.c_int), ("Cout", ctypes.c_int),
                ("act", ctypes.c_int), ("dtype", ctypes.c_int)]


class ccv3d_qcache_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("N", "C", "H", "W", "ring_slots", "format", "dtype")]


class CCV3DError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)} ({ccv3d_strerror(status)})")


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"libccv3d.so not built ({LIB_PATH}); run "
            "`python -m causal_conv3d_video_b200.build` (nvcc, sm_100a)")
    lib = ctypes.CDLL(LIB_PATH)
    vp, ip, i3 = ctypes.c_void_p, ctypes.POINTER(ctypes.c_int), ctypes.c_int * 3
    lib.ccv3d_plan.argtypes = [ctypes.POINTER(vp), ctypes.POINTER(ccv3d_desc)]
    lib.ccv3d_plan_intervals.argtypes = [vp, ip, ip, ip, ip, ip, ip]
    lib.ccv3d_plan_path.argtypes = [vp, ip, ip]
    lib.ccv3d_plan_path.restype = ctypes.c_int
    lib.ccv3d_forward.argtypes = [vp, vp, vp, vp, vp, vp, vp, ip, ip, ip, vp]
    lib.ccv3d_get_stats.argtypes = [vp, ctypes.POINTER(ccv3d_stats)]
    lib.ccv3d_get_status.argtypes = [vp]
    lib.ccv3d_destroy.argtypes = [vp]
    lib.ccv3d_destroy.restype = None
    lib.ccv3d_strerror.argtypes = [ctypes.c_int]
    lib.ccv3d_strerror.restype = ctypes.c_char_p
    lib.ccv3d_plan_kernel.argtypes = [vp]
    lib.ccv3d_plan_kernel.restype = ctypes.c_char_p
    lib.ccv3d_plan_tiling.argtypes = [vp, ip, ip, ip]
    lib.ccv3d_plan_tiling.restype = ctypes.c_int
    lib.ccv3d_plan_sizes.argtypes = [vp, ctypes.POINTER(ctypes.c_size_t),
                                     ctypes.POINTER(ctypes.c_size_t), ip]
    lib.ccv3d_selftest_wait_timeout.argtypes = [ctypes.c_uint64, vp]
    lib.ccv3d_quantize_u8.argtypes = [vp, ctypes.c_int, vp, ctypes.c_longlong, vp]
    lib.ccv3d_quantize_u8.restype = ctypes.c_int
    lib.ccv3d_forward_noalloc.argtypes = [ctypes.POINTER(ccv3d_desc), vp, vp, vp, vp, vp, vp,
                                          ip, ip, ip, vp]
    lib.ccv3d_get_status_stream.argtypes = [vp, vp]
    lib.ccv3d_selftest_bounds.argtypes = [vp]
    lib.ccv3d_selftest_bounds.restype = ctypes.c_int
    lib.ccv3d_noalloc_get_status.argtypes = [vp]
    lib.ccv3d_forward_ring.argtypes = [vp, vp, vp, ctypes.c_int, ctypes.c_int, vp, vp, vp,
                                       ip, ip, ip, vp, ip]
    c_int, c_size, p_size = ctypes.c_int, ctypes.c_size_t, ctypes.POINTER(ctypes.c_size_t)
    norm, point, qcache = (ctypes.POINTER(t) for t in (ccv3d_norm_desc, ccv3d_pointwise_desc,
                                                       ccv3d_qcache_desc))
    lib.ccv3d_norm_forward.argtypes = [norm] + [vp] * 10
    lib.ccv3d_norm_workspace.argtypes = [norm]
    lib.ccv3d_norm_workspace.restype = c_size
    lib.ccv3d_norm_backward.argtypes = [norm] + [vp] * 17 + [c_size, vp]
    lib.ccv3d_pointwise_workspace.argtypes = [point, p_size, p_size]
    lib.ccv3d_pointwise_forward.argtypes = [point] + [vp] * 7 + [c_size, vp]
    lib.ccv3d_pointwise_backward.argtypes = [point] + [vp] * 8 + [c_size, vp]
    lib.ccv3d_qcache_sizes.argtypes = [qcache, p_size, p_size]
    lib.ccv3d_qcache_write.argtypes = [qcache, vp, c_int, c_int, c_int, c_int, vp, vp, vp]
    lib.ccv3d_qcache_read.argtypes = [qcache, vp, vp, c_int, c_int, vp, vp]
    lib.ccv3d_forward_qring.argtypes = [vp, vp, qcache, vp, vp, c_int, vp, vp, vp, vp, ip, ip, ip,
                                        vp, ip]
    lib.ccv3d_block_get_status.argtypes = [vp]
    for f in ("ccv3d_norm_forward", "ccv3d_norm_backward", "ccv3d_pointwise_workspace",
              "ccv3d_pointwise_forward", "ccv3d_pointwise_backward", "ccv3d_qcache_sizes",
              "ccv3d_qcache_write", "ccv3d_qcache_read", "ccv3d_forward_qring",
              "ccv3d_block_get_status"):
        getattr(lib, f).restype = c_int
    for f in ("ccv3d_plan", "ccv3d_plan_intervals", "ccv3d_forward", "ccv3d_get_stats",
              "ccv3d_get_status", "ccv3d_plan_sizes", "ccv3d_selftest_wait_timeout",
              "ccv3d_forward_noalloc", "ccv3d_get_status_stream", "ccv3d_noalloc_get_status",
              "ccv3d_forward_ring"):
        getattr(lib, f).restype = ctypes.c_int
    del i3
    return lib


lib = _load()


def _ptr(t) -> int | None:
    """Device address of a tensor (or an int address); None for NULL."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(s) -> int | None:
    if s is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(s, int):
        return s
    return s.cuda_stream


def ccv3d_strerror(status: int) -> str:
    return lib.ccv3d_strerror(int(status)).decode()


class ccv3d_plan_t(ctypes.c_void_p):
    """A plan's handle, and the elements of its calls' tensors by name."""
    elements = None


def ccv3d_plan(desc: ccv3d_desc) -> ccv3d_plan_t:
    h = ccv3d_plan_t()
    rc = lib.ccv3d_plan(ctypes.byref(h), ctypes.byref(desc))
    if rc != 0:
        raise CCV3DError(rc, "ccv3d_plan")
    frame = desc.N * desc.H * desc.W * desc.Cin
    h.elements = {"x": frame * desc.T_x, "cache_buf": frame * desc.cache_len,
                  "w": desc.Cout * desc.kt * desc.kh * desc.kw * desc.Cin, "bias": desc.Cout,
                  "out": ccv3d_plan_sizes(h)["out_bytes"] // (2 if desc.dtype == CCV3D_BF16 else 4)}
    return h


def ccv3d_plan_intervals(plan) -> dict:
    T_o, H_o, W_o = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    d, lo, hi = (ctypes.c_int * 3)(), (ctypes.c_int * 3)(), (ctypes.c_int * 3)()
    rc = lib.ccv3d_plan_intervals(plan, ctypes.byref(T_o), ctypes.byref(H_o),
                                  ctypes.byref(W_o), d, lo, hi)
    if rc != 0:
        raise CCV3DError(rc, "ccv3d_plan_intervals")
    return {"T_o": T_o.value, "H_o": H_o.value, "W_o": W_o.value,
            "delta": list(d), "o_l": list(lo), "o_h": list(hi)}


def ccv3d_plan_path(plan):
    tm, tn = ctypes.c_int(), ctypes.c_int()
    tc = lib.ccv3d_plan_path(plan, ctypes.byref(tm), ctypes.byref(tn))
    return {"tc": bool(tc == 1), "tile_m": tm.value, "tile_n": tn.value}


def ccv3d_plan_kernel(plan) -> str:
    return lib.ccv3d_plan_kernel(plan).decode()


def ccv3d_plan_tiling(plan) -> dict:
    kb, st, g = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    rc = lib.ccv3d_plan_tiling(plan, ctypes.byref(kb), ctypes.byref(st), ctypes.byref(g))
    if rc not in (0, 2):
        raise CCV3DError(rc, "ccv3d_plan_tiling")
    return {"k_block": kb.value, "stages": st.value, "workspace_pairs": g.value}


def ccv3d_plan_sizes(plan):
    ob, nb, nf = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_int()
    rc = lib.ccv3d_plan_sizes(plan, ctypes.byref(ob), ctypes.byref(nb), ctypes.byref(nf))
    if rc != 0:
        raise CCV3DError(rc, "ccv3d_plan_sizes")
    return {"out_bytes": ob.value, "new_cache_bytes": nb.value, "new_cache_frames": nf.value}


def ccv3d_forward(plan, x, cache, w, bias, out, new_cache, stride, pad, dilation,
                  stream=None, check: bool = True) -> int:
    """One cached causal Conv3D call.  Tensors are device tensors in NTHWC
    physical order (contiguous, or channels_last_3d views) or int addresses.
    Raises CCV3DError on a refused call unless check=False (then returns the
    status code)."""
    s = (ctypes.c_int * 2)(*stride)
    p = (ctypes.c_int * 2)(*pad)
    d = (ctypes.c_int * 3)(*dilation)
    rc = lib.ccv3d_forward(plan, _ptr(x), _ptr(cache), _ptr(w), _ptr(bias), _ptr(out),
                           _ptr(new_cache), s, p, d, _stream(stream))
    if rc != 0 and check:
        raise CCV3DError(rc, "ccv3d_forward")
    return rc


def ccv3d_forward_ring(plan, x, ring, ring_slots: int, head: int, w, bias, out, stride, pad,
                       dilation, stream=None, check: bool = True):
    """The call with its cache in a ring buffer of ring_slots frames per batch
    entry (cache frame t at slot (head + t) % ring_slots).  Writes only the
    arriving frames of the new cache into the ring.  Returns (status,
    next_head); raises CCV3DError on a refused call unless check=False."""
    s = (ctypes.c_int * 2)(*stride)
    p = (ctypes.c_int * 2)(*pad)
    d = (ctypes.c_int * 3)(*dilation)
    nh = ctypes.c_int(-1)
    rc = lib.ccv3d_forward_ring(plan, _ptr(x), _ptr(ring), int(ring_slots), int(head), _ptr(w),
                                _ptr(bias), _ptr(out), s, p, d, _stream(stream),
                                ctypes.byref(nh))
    if rc != 0 and check:
        raise CCV3DError(rc, "ccv3d_forward_ring")
    return rc, nh.value


def ccv3d_forward_noalloc(desc: ccv3d_desc, x, cache, w, bias, out, new_cache, stride, pad,
                          dilation, stream=None, check: bool = True) -> int:
    """The no-allocation variant of ccv3d_forward: no plan, no device memory
    allocated by the library (its scratch is a fixed array inside the shared
    library, shared by all such calls on a device -- they must not overlap on
    the GPU).  For callers that may not allocate device memory."""
    s = (ctypes.c_int * 2)(*stride)
    p = (ctypes.c_int * 2)(*pad)
    d = (ctypes.c_int * 3)(*dilation)
    rc = lib.ccv3d_forward_noalloc(ctypes.byref(desc), _ptr(x), _ptr(cache), _ptr(w), _ptr(bias),
                                   _ptr(out), _ptr(new_cache), s, p, d, _stream(stream))
    if rc != 0 and check:
        raise CCV3DError(rc, "ccv3d_forward_noalloc")
    return rc


def ccv3d_get_stats(plan) -> dict:
    st = ccv3d_stats()
    rc = lib.ccv3d_get_stats(plan, ctypes.byref(st))
    if rc != 0:
        raise CCV3DError(rc, "ccv3d_get_stats")
    return {n: getattr(st, n) for n, _ in ccv3d_stats._fields_}


def ccv3d_get_status(plan) -> int:
    return lib.ccv3d_get_status(plan)


def ccv3d_get_status_stream(plan, stream=None) -> int:
    return lib.ccv3d_get_status_stream(plan, _stream(stream))


def ccv3d_noalloc_get_status(stream=None) -> int:
    return lib.ccv3d_noalloc_get_status(_stream(stream))


def ccv3d_destroy(plan) -> None:
    lib.ccv3d_destroy(plan)


def ccv3d_quantize_u8(x, out, stream=None, check: bool = True) -> int:
    """uint8 frames from decoded values on the device: out = trunc(clamp(
    fp32(x) * 255, 0, 255)), NaN -> 0.  x: a float32 or bfloat16 device
    tensor (any shape, contiguous); out: a uint8 device tensor of as many
    elements.  Raises CCV3DError on a refused call unless check=False."""
    import torch
    dt = {torch.float32: CCV3D_FP32, torch.bfloat16: CCV3D_BF16}.get(x.dtype)
    if dt is None or out.dtype != torch.uint8 or out.numel() != x.numel():
        raise ValueError("ccv3d_quantize_u8: x float32/bfloat16, out uint8 of x.numel()")
    if not (x.is_contiguous() and out.is_contiguous()):
        raise ValueError("ccv3d_quantize_u8: contiguous tensors only")
    rc = lib.ccv3d_quantize_u8(_ptr(x), dt, _ptr(out), x.numel(), _stream(stream))
    if rc != 0 and check:
        raise CCV3DError(rc, "ccv3d_quantize_u8")
    return rc


def ccv3d_selftest_wait_timeout(limit_ns: int, stream=None) -> int:
    return lib.ccv3d_selftest_wait_timeout(int(limit_ns), _stream(stream))


def ccv3d_selftest_bounds(stream=None) -> int:
    return lib.ccv3d_selftest_bounds(_stream(stream))


# ------------------------------------------- the operators around the convolution
# torch's types and the cheapest queries of the current device and stream,
# looked up at the first call (a call of a few microseconds is bound by this
# binding's own time)
_dtypes = _device_now = _stream_now = None


def _first_call():
    global _dtypes, _device_now, _stream_now
    import torch
    _device_now = torch.cuda.current_device
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    _stream_now = raw or (lambda dev: torch.cuda.current_stream(dev).cuda_stream)
    _dtypes = {CCV3D_BF16: torch.bfloat16, CCV3D_FP32: torch.float32, "uint8": torch.uint8}


def _refuse(where, name, t, n, want, device):
    if want is not None and t.dtype is not want:
        raise ValueError(f"{where}: {name} is {t.dtype}, not {want}")
    if n is not None and t.numel() != n:
        raise ValueError(f"{where}: {name} has {t.numel()} elements, not {n}")
    if not t.is_contiguous():
        raise ValueError(f"{where}: {name} is not contiguous")
    raise ValueError(f"{where}: {name} is on {t.device}, not on the current CUDA device {device}")


def _operands(where, dtype, stream, tensors, extra=()):
    """Device addresses of a call's buffers, then the stream's.  tensors: (name,
    tensor or address or None, elements) of the call's element type; extra:
    (name, tensor, elements, type) of others.  Tensors must be contiguous, of the
    type and size the call reads or writes, on the current CUDA device; raises
    ValueError otherwise.  Raw addresses are the caller's word."""
    if _dtypes is None:
        _first_call()
    want = _dtypes.get(dtype)
    out, device = [], None
    for name, t, n in tensors:
        if t is None or type(t) is int:
            out.append(t)
            continue
        d = t.get_device()
        if device is None:
            device = _device_now() if d >= 0 else -2
        if (d != device or t.numel() != n or not t.is_contiguous()
                or (t.dtype is not want and want is not None)):
            _refuse(where, name, t, n, want, device)
        out.append(t.data_ptr())
    for name, t, n, dt in extra:
        if t is None or type(t) is int:
            out.append(t)
            continue
        d = t.get_device()
        if device is None:
            device = _device_now() if d >= 0 else -2
        other = _dtypes.get(dt)
        if (d != device or (n is not None and t.numel() != n) or not t.is_contiguous()
                or (t.dtype is not other and other is not None)):
            _refuse(where, name, t, n, other, device)
        out.append(t.data_ptr())
    if stream is None:
        stream = _stream_now(_device_now() if device is None else device)
    elif type(stream) is not int:
        stream = stream.cuda_stream
    return out, stream


def _status(rc, where, check):
    if rc != 0 and check:
        raise CCV3DError(rc, where)
    return rc


def _bytes(where, ws, given):
    """Size of a workspace: a tensor of any type, None, or the `given` bytes at a
    raw address."""
    if ws is None:
        return 0
    if type(ws) is int:
        if given is None:
            raise ValueError(f"{where}: ws is a raw address, whose size ws_bytes has to say")
        return given
    return ws.numel() * ws.element_size()


def ccv3d_norm_workspace(desc: ccv3d_norm_desc) -> int:
    return lib.ccv3d_norm_workspace(ctypes.byref(desc))


def ccv3d_norm_forward(desc: ccv3d_norm_desc, h, b, gate, post_w, post_bias, pre_w, pre_bias,
                       h_out, y, stream=None, check: bool = True) -> int:
    """h_out = h + scale * gate * post(b); y = act(pre(h_out)).  Tensors as the
    C call's comment lists them (None for NULL).  Raises CCV3DError on a
    refused call unless check=False."""
    C = desc.C
    n = desc.rows * C
    gates = n // max(1, desc.gate_rows) if gate is not None else 0
    a, st = _operands("ccv3d_norm_forward", desc.dtype, stream, (
        ("h", h, n), ("b", b, n), ("gate", gate, gates), ("post_w", post_w, C),
        ("post_bias", post_bias, C), ("pre_w", pre_w, C), ("pre_bias", pre_bias, C),
        ("h_out", h_out, n), ("y", y, n)))
    return _status(lib.ccv3d_norm_forward(desc, *a, st), "ccv3d_norm_forward", check)


def ccv3d_norm_backward(desc: ccv3d_norm_desc, h_out, b, gate, post_w, post_bias, pre_w, pre_bias,
                        dy, dh_out, dh, db, dgate, dpost_w, dpost_bias, dpre_w, dpre_bias, ws,
                        stream=None, check: bool = True, ws_bytes: int | None = None) -> int:
    """Gradients of ccv3d_norm_forward (None for those not wanted); ws: a
    workspace of at least ccv3d_norm_workspace(desc) bytes (ws_bytes: the size of
    one given as a raw address)."""
    C = desc.C
    n = desc.rows * C
    gates = n // max(1, desc.gate_rows) if gate is not None else 0
    where = "ccv3d_norm_backward"
    a, st = _operands(where, desc.dtype, stream, (
        ("h_out", h_out, n), ("b", b, n), ("gate", gate, gates), ("post_w", post_w, C),
        ("post_bias", post_bias, C), ("pre_w", pre_w, C), ("pre_bias", pre_bias, C),
        ("dy", dy, n), ("dh_out", dh_out, n), ("dh", dh, n), ("db", db, n),
        ("dgate", dgate, gates), ("dpost_w", dpost_w, C), ("dpost_bias", dpost_bias, C),
        ("dpre_w", dpre_w, C), ("dpre_bias", dpre_bias, C)), (("ws", ws, None, None),))
    return _status(lib.ccv3d_norm_backward(desc, *a, _bytes(where, ws, ws_bytes), st), where, check)


def ccv3d_pointwise_workspace(desc: ccv3d_pointwise_desc):
    """(forward, backward) workspace bytes."""
    f, b = ctypes.c_size_t(), ctypes.c_size_t()
    _status(lib.ccv3d_pointwise_workspace(ctypes.byref(desc), ctypes.byref(f), ctypes.byref(b)),
            "ccv3d_pointwise_workspace", True)
    return f.value, b.value


def ccv3d_pointwise_forward(desc: ccv3d_pointwise_desc, x, w, bias, residual, out, pre, ws,
                            stream=None, check: bool = True, ws_bytes: int | None = None) -> int:
    """out = act(x w^T + bias) + residual; pre (None: not wanted) receives the
    argument of act.  ws_bytes: the size of a ws given as a raw address."""
    M, K, N = desc.pixels, desc.Cin, desc.Cout
    where = "ccv3d_pointwise_forward"
    a, st = _operands(where, desc.dtype, stream, (
        ("x", x, M * K), ("w", w, N * K), ("bias", bias, N), ("residual", residual, M * N),
        ("out", out, M * N), ("pre", pre, M * N)), (("ws", ws, None, None),))
    return _status(lib.ccv3d_pointwise_forward(desc, *a, _bytes(where, ws, ws_bytes), st), where,
                   check)


def ccv3d_pointwise_backward(desc: ccv3d_pointwise_desc, x, w, pre, dout, dx, dw, dbias, ws,
                             stream=None, check: bool = True, ws_bytes: int | None = None) -> int:
    """Gradients of ccv3d_pointwise_forward (None for those not wanted).  ws_bytes:
    the size of a ws given as a raw address."""
    M, K, N = desc.pixels, desc.Cin, desc.Cout
    where = "ccv3d_pointwise_backward"
    a, st = _operands(where, desc.dtype, stream, (
        ("x", x, M * K), ("w", w, N * K), ("pre", pre, M * N), ("dout", dout, M * N),
        ("dx", dx, M * K), ("dw", dw, N * K), ("dbias", dbias, N)), (("ws", ws, None, None),))
    return _status(lib.ccv3d_pointwise_backward(desc, *a, _bytes(where, ws, ws_bytes), st), where,
                   check)


def ccv3d_qcache_sizes(desc: ccv3d_qcache_desc):
    """(codes, scales) bytes."""
    c, s = ctypes.c_size_t(), ctypes.c_size_t()
    _status(lib.ccv3d_qcache_sizes(ctypes.byref(desc), ctypes.byref(c), ctypes.byref(s)),
            "ccv3d_qcache_sizes", True)
    return c.value, s.value


def _ring(desc, codes, scales):
    """The two buffers of a quantised ring, for _operands."""
    px = desc.N * desc.ring_slots * desc.H * desc.W
    C = desc.C
    return (("codes", codes, px * ((C + 1) // 2 if desc.format == 2 else C), "uint8"),
            ("scales", scales, px * ((C + 31) // 32), "uint8"))


def ccv3d_qcache_write(desc: ccv3d_qcache_desc, x, T_x: int, first: int, frames: int, slot: int,
                       codes, scales, stream=None, check: bool = True) -> int:
    """Quantise frames [first, first + frames) of x into ring slots from `slot` on."""
    n = desc.N * T_x * desc.H * desc.W * desc.C
    a, st = _operands("ccv3d_qcache_write", desc.dtype, stream, (("x", x, n),),
                      _ring(desc, codes, scales))
    return _status(lib.ccv3d_qcache_write(desc, a[0], T_x, first, frames, slot, a[1], a[2], st),
                   "ccv3d_qcache_write", check)


def ccv3d_qcache_read(desc: ccv3d_qcache_desc, codes, scales, head: int, frames: int, out,
                      stream=None, check: bool = True) -> int:
    """Read ring slots from `head` on back into `frames` dense frames."""
    n = desc.N * frames * desc.H * desc.W * desc.C
    a, st = _operands("ccv3d_qcache_read", desc.dtype, stream, (("out", out, n),),
                      _ring(desc, codes, scales))
    return _status(lib.ccv3d_qcache_read(desc, a[1], a[2], head, frames, a[0], st),
                   "ccv3d_qcache_read", check)


def ccv3d_forward_qring(plan, x, desc: ccv3d_qcache_desc, codes, scales, head: int, cache_buf, w,
                        bias, out, stride, pad, dilation, stream=None, check: bool = True):
    """ccv3d_forward_ring with the ring held in 8 or 4 bits.  Tensors have to be of the
    sizes that the plan was made for; cache_buf, a scratch that modules may share,
    may be larger.  (A plan given as a raw handle is the caller's word for them.)
    Returns (status, next_head)."""
    dt, sizes = desc.dtype, getattr(plan, "elements", None)
    for name, t in (("x", x), ("cache_buf", cache_buf), ("w", w), ("bias", bias), ("out", out)):
        if sizes and t is not None and type(t) is not int:
            n = t.numel()
            if n < sizes[name] or (n > sizes[name] and name != "cache_buf"):
                raise ValueError(f"forward_qring: {name} has {n} elements, not {sizes[name]}")
    a, st = _operands("ccv3d_forward_qring", dt, stream, (), (
        ("x", x, None, dt), *_ring(desc, codes, scales), ("cache_buf", cache_buf, None, dt),
        ("w", w, None, dt), ("bias", bias, None, dt), ("out", out, None, dt)))
    s, p, d = (ctypes.c_int * 2)(*stride), (ctypes.c_int * 2)(*pad), (ctypes.c_int * 3)(*dilation)
    nh = ctypes.c_int(-1)
    rc = lib.ccv3d_forward_qring(plan, a[0], desc, a[1], a[2], int(head), a[3], a[4], a[5], a[6],
                                 s, p, d, st, ctypes.byref(nh))
    return _status(rc, "ccv3d_forward_qring", check), nh.value


def ccv3d_block_get_status(stream=None) -> int:
    return lib.ccv3d_block_get_status(_stream(stream))


# ---------------------------------------------------------------- helpers
def _dtype_code(dtype):
    return {"bf16": CCV3D_BF16, "fp32": CCV3D_FP32}[dtype]


def make_norm_desc(*, rows, C, pre="rms", post="none", act="none", eps=1e-6, scale=1.0,
                   gate_rows=0, dtype="bf16") -> ccv3d_norm_desc:
    """gate_rows: consecutive rows that share a row of the gate (0: no gate)."""
    return ccv3d_norm_desc(rows, C, NORM_KINDS[pre], NORM_KINDS[post], ACTS[act], eps, scale,
                           gate_rows, _dtype_code(dtype))


def make_pointwise_desc(*, pixels, Cin, Cout, act="none", dtype="bf16") -> ccv3d_pointwise_desc:
    return ccv3d_pointwise_desc(pixels, Cin, Cout, ACTS[act], _dtype_code(dtype))


def make_qcache_desc(*, N, H, W, C, ring_slots, format="int8", dtype="bf16") -> ccv3d_qcache_desc:
    return ccv3d_qcache_desc(N, C, H, W, ring_slots, QFORMATS[format], _dtype_code(dtype))


def alloc_workspace(nbytes: int, device="cuda"):
    """A workspace of that many bytes (None for 0)."""
    import torch
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


def alloc_qcache(desc: ccv3d_qcache_desc, device="cuda"):
    """(codes, scales) of a quantised ring cache, empty."""
    import torch
    return tuple(torch.zeros(n, dtype=torch.uint8, device=device)
                 for n in ccv3d_qcache_sizes(desc))


def make_desc(*, N, Cin, Cout, H, W, T_x, cache_len, kt=3, kh=3, kw=3,
              pad_t_base=None, cache_keep=None, stride=(1, 1), pad=(1, 1),
              dilation=(1, 1, 1), dtype="bf16", has_bias=True, stride_t=1,
              groups=1) -> ccv3d_desc:
    if pad_t_base is None:
        pad_t_base = dilation[0] * (kt - 1)
    if cache_keep is None:
        cache_keep = pad_t_base
    return ccv3d_desc(N, Cin, Cout, kt, kh, kw, H, W, T_x, cache_len, pad_t_base,
                      cache_keep, stride_t, stride[0], stride[1], pad[0], pad[1],
                      dilation[0], dilation[1], dilation[2], groups,
                      CCV3D_BF16 if dtype == "bf16" else CCV3D_FP32, int(bool(has_bias)))


def desc_for(conv) -> ccv3d_desc:
    """Descriptor for a workloads.Conv signature."""
    return make_desc(N=conv.N, Cin=conv.Cin, Cout=conv.Cout, H=conv.H, W=conv.W,
                     T_x=conv.T_x, cache_len=conv.cache_len, kt=conv.kt, kh=conv.kh,
                     kw=conv.kw, pad_t_base=conv.pad_t_base, cache_keep=conv.cache_keep,
                     stride=conv.stride, pad=conv.pad, dilation=conv.dilation,
                     dtype=conv.dtype, has_bias=conv.has_bias, stride_t=conv.stride_t)


class Plan:
    """Owning wrapper of a ccv3d plan handle (destroyed with the object)."""

    def __init__(self, desc: ccv3d_desc):
        self.desc = desc
        self.handle = ccv3d_plan(desc)
        self.intervals = ccv3d_plan_intervals(self.handle)
        self.sizes = ccv3d_plan_sizes(self.handle)
        self.path = ccv3d_plan_path(self.handle)
        self.kernel = ccv3d_plan_kernel(self.handle)
        self.tiling = ccv3d_plan_tiling(self.handle)

    @property
    def stride(self):
        return (self.desc.stride_h, self.desc.stride_w)

    @property
    def pad(self):
        return (self.desc.pad_h, self.desc.pad_w)

    @property
    def dilation(self):
        return (self.desc.dil_t, self.desc.dil_h, self.desc.dil_w)

    def out_shape(self):
        d, iv = self.desc, self.intervals
        return (d.N, iv["T_o"], iv["H_o"], iv["W_o"], d.Cout)

    def new_cache_shape(self):
        d = self.desc
        return (d.N, self.sizes["new_cache_frames"], d.H, d.W, d.Cin)

    def forward(self, x, cache, w, bias, out, new_cache, stream=None):
        return ccv3d_forward(self.handle, x, cache, w, bias, out, new_cache, self.stride,
                             self.pad, self.dilation, stream)

    def forward_ring(self, x, ring, ring_slots, head, w, bias, out, stream=None):
        """Ring-buffer cache call; returns the head of the new cache."""
        return ccv3d_forward_ring(self.handle, x, ring, ring_slots, head, w, bias, out,
                                  self.stride, self.pad, self.dilation, stream)[1]

    def forward_qring(self, x, desc, codes, scales, head, cache_buf, w, bias, out, stream=None):
        """Call with its ring cache in 8 or 4 bits; returns the head of the new cache."""
        return ccv3d_forward_qring(self.handle, x, desc, codes, scales, head, cache_buf, w, bias,
                                   out, self.stride, self.pad, self.dilation, stream)[1]

    def ring_writes(self):
        """Frames of x a ring-buffer call writes into the ring."""
        return min(self.sizes["new_cache_frames"], self.desc.T_x)

    def alloc_outputs(self, device="cuda"):
        import torch
        dt = torch.bfloat16 if self.desc.dtype == CCV3D_BF16 else torch.float32
        out = torch.empty(self.out_shape(), dtype=dt, device=device)
        nc = (torch.empty(self.new_cache_shape(), dtype=dt, device=device)
              if self.sizes["new_cache_frames"] > 0 else None)
        return out, nc

    def stats(self):
        return ccv3d_get_stats(self.handle)

    def status(self):
        return ccv3d_get_status(self.handle)

    def status_stream(self, stream=None):
        return ccv3d_get_status_stream(self.handle, stream)

    def close(self):
        if getattr(self, "handle", None) is not None:
            ccv3d_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
