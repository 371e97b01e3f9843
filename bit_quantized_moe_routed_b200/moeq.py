"""Python binding of libmoeq (ctypes; argument marshalling only).

Every step of the layer runs in the CUDA library; this module only turns
torch tensors / numpy arrays into pointers, sizes and the current CUDA
stream.  It raises at import time when ``libmoeq.so`` is missing: there is
no fallback implementation.
"""
from __future__ import annotations

import ctypes as C
import functools
import os
import struct

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoeq.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python -m bit_quantized_moe_routed_b200.build` "
        "(the layer has no non-CUDA implementation)")

_lib = C.CDLL(LIB_PATH)

OK, INVALID_ARGUMENT, UNSUPPORTED, OUT_OF_MEMORY, CUDA, NOT_UPLOADED, ROUTE_OUT_OF_RANGE, TIMEOUT = range(8)
FMT = {"mxfp4": 0, "vq13": 1, "vq13r8": 2, "gvq1": 3, "gvq1r8": 4}
ACT = {"f32": 0, "bf16": 1}
GATE, UP, DOWN = 0, 1, 2

# every symbol the header declares
EXPORTS = ("moeq_layer_create", "moeq_upload_weights", "moeq_forward", "moeq_forward_host",
           "moeq_forward_profiled", "moeq_route", "moeq_dequant", "moeq_layer_status",
           "moeq_status_string", "moeq_layer_destroy", "moeq_kernel_launches", "moeq_route_noalloc",
           "moeq_router_upload", "moeq_router", "moeq_forward_routed", "moeq_vq_encode",
           "moeq_quant_i8", "moeq_matmul_i8", "moeq_glu_i8", "moeq_i8_workspace", "moeq_glu",
           "moeq_glu_backward", "moeq_glu_workspace", "moeq_dense_status")
SCORE = {"sigmoid": 0, "softmax": 1}


class LayerDesc(C.Structure):
    _fields_ = [("hidden", C.c_int32), ("inter", C.c_int32), ("n_experts", C.c_int32),
                ("top_k", C.c_int32), ("max_tokens", C.c_int32), ("fmt", C.c_int32),
                ("act", C.c_int32), ("device", C.c_int32)]


class Weights(C.Structure):
    _fields_ = [("codes", C.c_void_p * 3), ("scales", C.c_void_p * 3), ("idx13", C.c_void_p * 3),
                ("idx8", C.c_void_p * 3), ("book13", C.c_void_p), ("book8", C.c_void_p),
                ("gain", C.c_void_p * 3), ("code12", C.c_void_p * 3), ("hi1", C.c_void_p * 3),
                ("gbook13", C.c_void_p), ("gbook8", C.c_void_p), ("gscale", C.c_float * 2)]


_lib.moeq_layer_create.argtypes = [C.POINTER(LayerDesc), C.POINTER(C.c_void_p)]
_lib.moeq_upload_weights.argtypes = [C.c_void_p, C.POINTER(Weights), C.c_void_p]
_lib.moeq_forward.argtypes = [C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_int32, C.c_void_p, C.c_void_p]
_lib.moeq_forward_host.argtypes = [C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_int32, C.c_void_p,
                                   C.c_void_p]
_lib.moeq_forward_profiled.argtypes = [C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_int32, C.c_void_p,
                                       C.c_void_p, C.POINTER(C.c_void_p)]
_lib.moeq_route.argtypes = [C.c_void_p, C.c_void_p, C.c_int32, C.c_void_p, C.c_void_p, C.c_void_p]
_lib.moeq_route_noalloc.argtypes = [C.c_void_p, C.c_int32, C.c_int32, C.c_int32, C.c_void_p, C.c_void_p, C.c_void_p]
_lib.moeq_dequant.argtypes = [C.c_void_p, C.c_int32, C.c_int32, C.c_void_p, C.c_void_p]
_lib.moeq_router_upload.argtypes = [C.c_void_p, C.c_void_p, C.c_int32, C.c_void_p]
_lib.moeq_router.argtypes = [C.c_void_p, C.c_void_p, C.c_int32, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p]
_lib.moeq_forward_routed.argtypes = [C.c_void_p, C.c_void_p, C.c_int32, C.c_void_p, C.c_void_p, C.c_void_p,
                                     C.c_void_p]
_lib.moeq_vq_encode.argtypes = [C.c_void_p, C.c_int32, C.c_int32, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p,
                                C.c_void_p, C.c_void_p, C.c_void_p]
_lib.moeq_layer_status.argtypes = [C.c_void_p, C.c_int32]
_lib.moeq_status_string.argtypes = [C.c_int]
_lib.moeq_status_string.restype = C.c_char_p
_lib.moeq_layer_destroy.argtypes = [C.c_void_p]
_lib.moeq_layer_destroy.restype = None
_lib.moeq_kernel_launches.argtypes = [C.c_void_p]
_lib.moeq_kernel_launches.restype = C.c_int64
for _f in ("moeq_layer_create", "moeq_upload_weights", "moeq_forward", "moeq_forward_host", "moeq_dequant",
           "moeq_layer_status", "moeq_forward_profiled", "moeq_route", "moeq_route_noalloc",
           "moeq_router_upload", "moeq_router", "moeq_forward_routed", "moeq_vq_encode"):
    getattr(_lib, _f).restype = C.c_int


# the argument structs of the dense operators, packed as the C compiler lays
# them out (native sizes and alignment)
I8_ARGS = struct.Struct("@4i Pq P 2P 2q 2P Pq Pq")      # moeq_i8_args
GLU_ARGS = struct.Struct("@4i Pq 2P 2q P Pq Pq Pq 2P 2q Pq")   # moeq_glu_args
_lib.moeq_quant_i8.argtypes = [C.c_void_p, C.c_int32, C.c_int32, C.c_int32, C.c_int64, C.c_void_p, C.c_int64,
                               C.c_void_p, C.c_void_p]
for _f in ("moeq_matmul_i8", "moeq_glu_i8", "moeq_glu", "moeq_glu_backward"):
    getattr(_lib, _f).argtypes = [C.c_char_p, C.c_void_p]
for _f in ("moeq_i8_workspace", "moeq_glu_workspace"):
    getattr(_lib, _f).argtypes = [C.c_char_p, C.c_int32]
    getattr(_lib, _f).restype = C.c_int64
_lib.moeq_dense_status.argtypes = [C.c_int32]
for _f in ("moeq_quant_i8", "moeq_matmul_i8", "moeq_glu_i8", "moeq_glu", "moeq_glu_backward", "moeq_dense_status"):
    getattr(_lib, _f).restype = C.c_int


class MoeqError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {status_string(code)} ({code})")


def status_string(code: int) -> str:
    return _lib.moeq_status_string(int(code)).decode()


def lib():
    return _lib


def _check(code: int, what: str):
    if code != OK:
        raise MoeqError(code, what)


def _stream_ptr(stream):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return C.c_void_p(s.cuda_stream)


def _host(a, dtype):
    if a is None:
        return None, None
    a = np.ascontiguousarray(a, dtype=dtype)
    return a, a.ctypes.data


def route_noalloc(topk_ids, n_experts, offsets_out, perm_out, stream=None):
    """moeq_route_noalloc: the route/bucket step without a layer and without
    any device allocation.  topk_ids int32 cuda [T][k]; offsets_out int32
    cuda [n_experts+1] and perm_out int32 cuda [T*k] are the caller's and
    are filled as by Layer.route.  The library's fixed scratch is shared by
    every call on a device: calls that overlap on the GPU race."""
    T, k = topk_ids.shape
    _check(_lib.moeq_route_noalloc(C.c_void_p(topk_ids.data_ptr()), T, k, n_experts,
                                   C.c_void_p(offsets_out.data_ptr()), C.c_void_p(perm_out.data_ptr()),
                                   _stream_ptr(stream)), "moeq_route_noalloc")


def vq_encode(w, book13, book8=None, gain=None, col_weight=None, stream=None):
    """moeq_vq_encode on cuda tensors: w float32 [N][K]; book13 / book8
    bf16 bit patterns (int16 or uint16 tensors) [8192][8] / [256][8]; gain
    f16 bit patterns [N] or None; col_weight float32 [K] or None.  Returns
    (idx13 uint8 [N][K*13/64], idx8 uint8 [N][K/8] or None)."""
    import torch
    N, K = w.shape
    idx13 = torch.empty((N, K * 13 // 64), dtype=torch.uint8, device=w.device)
    idx8 = torch.empty((N, K // 8), dtype=torch.uint8, device=w.device) if book8 is not None else None

    def p(t):
        return C.c_void_p(t.data_ptr() if t is not None else 0)
    _check(_lib.moeq_vq_encode(p(w), N, K, p(gain), p(col_weight), p(book13), p(book8), p(idx13), p(idx8),
                               _stream_ptr(stream)), "moeq_vq_encode")
    return idx13, idx8


# The dense operators are called once a layer and step, some of them for a
# few microseconds of device work: their wrappers build messages only when
# they raise, ask for the workspace's size only when one is needed, and give
# torch's allocations their sizes one by one (half the time of a tuple).
def _bad(what):
    raise MoeqError(INVALID_ARGUMENT, what)


def _enter(t, stream, name):
    """(device index, raw stream) of a call on the current stream of t's
    device, which is the current device; or (device index, None): the call is
    to be made again inside _on(t, stream)."""
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        _bad(f"{name}: a cuda tensor is needed")
    dev = t.get_device()
    if stream is not None:
        if stream.device_index != dev:
            _bad(f"{name}: stream on {stream.device}, tensor on {t.device}")
        return dev, None
    if torch._C._cuda_getDevice() != dev:
        return dev, None
    return dev, torch._C._cuda_getCurrentRawStream(dev)


def _on(dev, stream):
    """Context of a call on ``stream`` (or the current stream of device
    ``dev``): allocations made in it belong to that stream."""
    import torch
    return torch.cuda.stream(stream) if stream is not None else torch.cuda.device(dev)


def _act(t, what):
    """moeq_dtype of a tensor."""
    import torch
    if t.dtype is torch.bfloat16:
        return 1
    if t.dtype is not torch.float32:
        _bad(f"{what}: dtype {t.dtype}")
    return 0


def _ld(t, rows, cols, dtype, dev, what):
    """Row stride of a 2-D cuda tensor with unit column stride, checked
    against the shape, dtype and device it must have."""
    if t.dtype is not dtype or t.shape != (rows, cols) or t.get_device() != dev:
        _bad(f"{what}: {t.dtype} {tuple(t.shape)} on {t.device}, need {dtype} {(rows, cols)} on cuda:{dev}")
    if t.is_contiguous():
        return cols
    rs, cs = t.stride()
    if cs != 1 and cols > 1:
        _bad(f"{what}: column stride {cs}")
    return rs if rows > 1 else max(rs, cols)


def _vec(t, n, dev, what):
    import torch
    if t.dtype is not torch.float32 or t.shape != (n,) or t.get_device() != dev or not t.is_contiguous():
        _bad(f"{what}: need contiguous float32 ({n},) on cuda:{dev}")
    return t.data_ptr()


def _call(run, query, which, args, layout, workspace, t, s, name):
    """One call; ``args`` lacks the workspace's address and size.  Without a
    workspace the call is tried as it is (a call that lacks one is refused
    before any work); where one is needed it is allocated on the call's
    stream."""
    if workspace is None:
        code = run(layout.pack(*args, 0, 0), s)
        if code == OK:
            return
        n = query(layout.pack(*args, 0, 0), which) if code == INVALID_ARGUMENT else 0
        if n <= 0:
            raise MoeqError(code, name)
        import torch
        workspace = torch.empty(n, dtype=torch.uint8, device=t.device)
    elif workspace.get_device() != t.get_device() or not workspace.is_contiguous():
        _bad(f"{name}: workspace is not contiguous on {t.device}")
    _check(run(layout.pack(*args, workspace.data_ptr(), workspace.numel() * workspace.element_size()), s), name)


def quant_i8(x, q=None, scale=None, stream=None):
    """moeq_quant_i8: rows of x (float32 or bfloat16 [M][K], unit column
    stride) to (q int8 [M][K], scale float32 [M]), x ~ q * scale[:, None].  A
    q made here starts its rows on multiples of 16 bytes (a view of a wider
    buffer where K is not one), as the products take it without a copy."""
    import torch
    dev, s = _enter(x, stream, "quant_i8")
    if s is None:
        with _on(dev, stream):
            return quant_i8(x, q, scale)
    if x.dim() != 2:
        _bad("quant_i8: x is not 2-D")
    M, K = x.shape
    if q is None:
        ldq = (K + 15) // 16 * 16
        q = torch.empty(M, ldq, dtype=torch.int8, device=x.device)
        if ldq != K:
            q = q.as_strided((M, K), (ldq, 1))
    else:
        ldq = _ld(q, M, K, torch.int8, dev, "quant_i8: q")
    if scale is None:
        scale = torch.empty(M, dtype=torch.float32, device=x.device)
    code = _lib.moeq_quant_i8(x.data_ptr(), _act(x, "quant_i8: x"), M, K, _ld(x, M, K, x.dtype, dev, "quant_i8: x"),
                              q.data_ptr(), ldq, _vec(scale, M, dev, "quant_i8: scale"), s)
    if code:
        _check(code, "moeq_quant_i8")
    return q, scale


def _i8(name, run, n_w, xq, xs, w0, s0, w1, s1, out, dtype, workspace, dev, s):
    import torch
    if xq.dim() != 2 or w0.dim() != 2:
        _bad(f"{name}: operands are not 2-D")
    T, K = xq.shape
    N = w0.shape[0]
    i8 = torch.int8
    if out is None:
        if dtype not in ACT:
            _bad(f"{name}: dtype {dtype!r}")
        act, ldo = ACT[dtype], N
        out = torch.empty(T, N, dtype=torch.bfloat16 if act else torch.float32, device=xq.device)
    else:
        act, ldo = _act(out, name), _ld(out, T, N, out.dtype, dev, name)
    ldx, px = _ld(xq, T, K, i8, dev, name), _vec(xs, T, dev, name)
    ld0, p0 = _ld(w0, N, K, i8, dev, name), _vec(s0, N, dev, name)
    a1 = ld1 = p1 = 0
    if w1 is not None:
        a1, ld1, p1 = w1.data_ptr(), _ld(w1, N, K, i8, dev, name), _vec(s1, N, dev, name)
    _call(run, _lib.moeq_i8_workspace, n_w,
          (T, K, N, act, xq.data_ptr(), ldx, px, w0.data_ptr(), a1, ld0, ld1, p0, p1, out.data_ptr(), ldo), I8_ARGS,
          workspace, xq, s, name)
    return out


def matmul_i8(xq, xs, wq, ws, out=None, dtype="bf16", workspace=None, stream=None):
    """moeq_matmul_i8: (xq wq^T) xs[:, None] ws with xq int8 [T][K], wq int8
    [N][K], xs float32 [T], ws float32 [N]; [T][N] in ``dtype`` ("bf16" or
    "f32"), or into ``out``."""
    dev, s = _enter(xq, stream, "matmul_i8")
    if s is None:
        with _on(dev, stream):
            return matmul_i8(xq, xs, wq, ws, out, dtype, workspace)
    return _i8("matmul_i8", _lib.moeq_matmul_i8, 1, xq, xs, wq, ws, None, None, out, dtype, workspace, dev, s)


def glu_i8(xq, xs, w_gate, s_gate, w_up, s_up, out=None, dtype="bf16", workspace=None, stream=None):
    """moeq_glu_i8: silu(G) * U with G, U the products of xq with the int8
    weights [N][K] of both projections, as matmul_i8."""
    dev, s = _enter(xq, stream, "glu_i8")
    if s is None:
        with _on(dev, stream):
            return glu_i8(xq, xs, w_gate, s_gate, w_up, s_up, out, dtype, workspace)
    return _i8("glu_i8", _lib.moeq_glu_i8, 2, xq, xs, w_gate, s_gate, w_up, s_up, out, dtype, workspace, dev, s)


def _glu_common(x, w_gate, w_up, gu, dev, what):
    if x.dim() != 2 or w_gate.dim() != 2:
        _bad(f"{what}: operands are not 2-D")
    T, H = x.shape
    N = w_gate.shape[0]
    dt = x.dtype
    act = _act(x, what)
    pgu = 0
    if gu is not None:
        if gu.dtype is not dt or gu.shape != (2, T, N) or gu.get_device() != dev or not gu.is_contiguous():
            _bad(f"{what}: gu is not a contiguous {dt} {(2, T, N)} on cuda:{dev}")
        pgu = gu.data_ptr()
    return T, H, N, dt, (T, H, N, act, x.data_ptr(), _ld(x, T, H, dt, dev, what), w_gate.data_ptr(), w_up.data_ptr(),
                         _ld(w_gate, N, H, dt, dev, what), _ld(w_up, N, H, dt, dev, what), pgu)


def glu(x, w_gate, w_up, save=False, out=None, gu=None, workspace=None, stream=None):
    """moeq_glu: h = silu(x w_gate^T) * (x w_up^T), [T][N], for x [T][H] and
    weights [N][H] (float32 or bfloat16, unit column stride).  With ``save``
    (or a ``gu`` buffer [2][T][N]) returns (h, gu) with both projections kept
    for glu_backward."""
    dev, s = _enter(x, stream, "glu")
    if s is None:
        with _on(dev, stream):
            return glu(x, w_gate, w_up, save, out, gu, workspace)
    if save and gu is None and x.dim() == 2 and w_gate.dim() == 2:
        gu = x.new_empty(2, x.shape[0], w_gate.shape[0])
    T, H, N, dt, head = _glu_common(x, w_gate, w_up, gu, dev, "glu")
    if out is None:
        out, ldh = x.new_empty(T, N), N
    else:
        ldh = _ld(out, T, N, dt, dev, "glu: out")
    _call(_lib.moeq_glu, _lib.moeq_glu_workspace, 0, head + (out.data_ptr(), ldh, 0, 0, 0, 0, 0, 0, 0, 0), GLU_ARGS,
          workspace, x, s, "glu")
    return out if gu is None else (out, gu)


def glu_backward(dh, x, w_gate, w_up, gu=None, dx=None, dw_gate=None, dw_up=None, need_dx=True, need_dw=True,
                 workspace=None, stream=None):
    """moeq_glu_backward: (dx [T][H], dw_gate [N][H], dw_up [N][H]) for the
    gradient dh [T][N] of glu's result; ``gu`` as kept by glu, or None to
    compute the projections again.  Gradients left out (``need_dx``,
    ``need_dw``) come back as None."""
    import torch
    what = "glu_backward"
    dev, s = _enter(dh, stream, what)
    if s is None:
        with _on(dev, stream):
            return glu_backward(dh, x, w_gate, w_up, gu, dx, dw_gate, dw_up, need_dx, need_dw, workspace)
    T, H, N, dt, head = _glu_common(x, w_gate, w_up, gu, dev, what)
    if not (need_dx or dx is None) or not (need_dw or (dw_gate is None and dw_up is None)):
        _bad(f"{what}: a buffer for a gradient that is left out")
    if not (need_dx or need_dw):
        _bad(f"{what}: no gradient asked for")
    pdx = lddx = pg = pu = ldg = ldu = 0
    if need_dx:
        if dx is None:
            dx = x.new_empty(T, H)
        pdx, lddx = dx.data_ptr(), _ld(dx, T, H, dt, dev, what)
    if need_dw:
        if dw_gate is None:
            dw_gate = x.new_empty(N, H)
        if dw_up is None:
            dw_up = x.new_empty(N, H)
        pg, pu = dw_gate.data_ptr(), dw_up.data_ptr()
        ldg, ldu = _ld(dw_gate, N, H, dt, dev, what), _ld(dw_up, N, H, dt, dev, what)
    args = head + (0, 0, dh.data_ptr(), _ld(dh, T, N, dt, dev, what), pdx, lddx, pg, pu, ldg, ldu)
    if workspace is None:
        n = _lib.moeq_glu_workspace(GLU_ARGS.pack(*args, 0, 0), 1)
        if n < 0:
            _bad(what)
        workspace = torch.empty(n, dtype=torch.uint8, device=x.device)
    _call(_lib.moeq_glu_backward, _lib.moeq_glu_workspace, 1, args, GLU_ARGS, workspace, x, s, what)
    return dx, dw_gate, dw_up


def dense_status(clear=False) -> int:
    """moeq_dense_status: the current device's status word of the dense operators."""
    return int(_lib.moeq_dense_status(1 if clear else 0))


class Layer:
    """One compressed-expert MoE layer owned by libmoeq on one CUDA device."""

    def __init__(self, hidden, inter, n_experts, top_k, max_tokens, fmt="mxfp4", act="bf16", device=0):
        self.desc = LayerDesc(hidden, inter, n_experts, top_k, max_tokens, FMT[fmt], ACT[act], device)
        self.fmt, self.act, self.device = fmt, act, device
        self.H, self.I, self.E, self.k, self.max_tokens = hidden, inter, n_experts, top_k, max_tokens
        h = C.c_void_p()
        _check(_lib.moeq_layer_create(C.byref(self.desc), C.byref(h)), "moeq_layer_create")
        self._h = h

    @classmethod
    def for_cfg(cls, cfg, max_tokens=None, device=0):
        return cls(cfg.H, cfg.I, cfg.E, cfg.k, max_tokens or cfg.T, cfg.fmt, cfg.act, device)

    @property
    def handle(self):
        return self._h

    def close(self):
        if getattr(self, "_h", None) and self._h.value:
            _lib.moeq_layer_destroy(self._h)
            self._h = C.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def upload(self, w, stream=None):
        """``w``: host arrays with the attributes codes, scales, idx13, idx8,
        gain, code12, hi1 (per-projection lists), book13, book8 (bf16),
        gbook13, gbook8 (E4M3) and gscale, logical layout; missing
        attributes count as absent."""
        ws = Weights()
        keep = []
        for p in range(3):
            for name, dt in (("codes", np.uint8), ("scales", np.uint8), ("idx13", np.uint8),
                             ("idx8", np.uint8), ("gain", np.uint16), ("code12", np.uint8), ("hi1", np.uint8)):
                arrs = getattr(w, name, None)
                arr, ptr = _host(arrs[p] if arrs is not None else None, dt)
                keep.append(arr)
                getattr(ws, name)[p] = ptr
        for name, dt in (("book13", np.uint16), ("book8", np.uint16), ("gbook13", np.uint8), ("gbook8", np.uint8)):
            arr, ptr = _host(getattr(w, name, None), dt)
            keep.append(arr)
            setattr(ws, name, ptr)
        gs = getattr(w, "gscale", None)
        if gs is not None:
            ws.gscale[0], ws.gscale[1] = float(gs[0]), float(gs[1])
        _check(_lib.moeq_upload_weights(self._h, C.byref(ws), _stream_ptr(stream)), "moeq_upload_weights")
        del keep

    def forward(self, x, topk_ids, topk_w, out=None, stream=None):
        """x: cuda tensor [T][H] (float32 or bfloat16 per ``act``); topk_ids
        int32 [T][k]; topk_w float32 [T][k]; returns ``out`` [T][H]."""
        import torch
        T = x.shape[0]
        for t in (x, topk_ids, topk_w):
            assert t.is_cuda and t.is_contiguous()
        assert topk_ids.dtype == torch.int32 and topk_w.dtype == torch.float32
        if out is None:
            out = torch.empty_like(x)
        _check(_lib.moeq_forward(self._h, C.c_void_p(x.data_ptr()), C.c_void_p(topk_ids.data_ptr()),
                                 C.c_void_p(topk_w.data_ptr()), T, C.c_void_p(out.data_ptr()),
                                 _stream_ptr(stream)), "moeq_forward")
        return out

    def forward_profiled(self, x, topk_ids, topk_w, out, events, stream=None):
        """moeq_forward recording 5 torch.cuda.Event objects at its phase
        boundaries (before; after route; after gate/up; after down; end)."""
        assert len(events) == 5
        evs = (C.c_void_p * 5)(*[C.c_void_p(e.cuda_event) for e in events])
        _check(_lib.moeq_forward_profiled(self._h, C.c_void_p(x.data_ptr()), C.c_void_p(topk_ids.data_ptr()),
                                          C.c_void_p(topk_w.data_ptr()), x.shape[0], C.c_void_p(out.data_ptr()),
                                          _stream_ptr(stream), evs), "moeq_forward_profiled")
        return out

    def route(self, topk_ids, stream=None):
        """(offsets int32 [E+1], perm int32 [T*k]) cuda tensors; only the
        first offsets[E] entries of perm are defined."""
        import torch
        T = topk_ids.shape[0]
        offsets = torch.empty(self.E + 1, dtype=torch.int32, device=topk_ids.device)
        perm = torch.full((T * self.k,), -1, dtype=torch.int32, device=topk_ids.device)
        _check(_lib.moeq_route(self._h, C.c_void_p(topk_ids.data_ptr()), T, C.c_void_p(offsets.data_ptr()),
                               C.c_void_p(perm.data_ptr()), _stream_ptr(stream)), "moeq_route")
        return offsets, perm

    def forward_host(self, x, topk_ids, topk_w, out=None, stream=None):
        """Host (numpy / CPU tensor) buffers in and out; synchronous."""
        x = np.ascontiguousarray(x)
        ids = np.ascontiguousarray(topk_ids, dtype=np.int32)
        w = np.ascontiguousarray(topk_w, dtype=np.float32)
        if out is None:
            out = np.empty_like(x)
        _check(_lib.moeq_forward_host(self._h, x.ctypes.data, ids.ctypes.data, w.ctypes.data, x.shape[0],
                                      out.ctypes.data, _stream_ptr(stream)), "moeq_forward_host")
        return out

    def forward_host_ptr(self, x_ptr, ids_ptr, w_ptr, T, out_ptr, stream=None):
        """moeq_forward_host on raw host pointers (pinned buffers)."""
        _check(_lib.moeq_forward_host(self._h, C.c_void_p(x_ptr), C.c_void_p(ids_ptr), C.c_void_p(w_ptr), T,
                                      C.c_void_p(out_ptr), _stream_ptr(stream)), "moeq_forward_host")

    def dequant(self, expert, proj, out=None, stream=None):
        import torch
        N, K = (self.I, self.H) if proj in (GATE, UP) else (self.H, self.I)
        if out is None:
            out = torch.empty((N, K), dtype=torch.float32, device=f"cuda:{self.device}")
        _check(_lib.moeq_dequant(self._h, expert, proj, C.c_void_p(out.data_ptr()), _stream_ptr(stream)),
               "moeq_dequant")
        return out

    def router_upload(self, wr, score="sigmoid", stream=None):
        """Router matrix ``wr``: host float32 [E][H]; ``score``: "sigmoid" or "softmax"."""
        wr = np.ascontiguousarray(wr, dtype=np.float32)
        assert wr.shape == (self.E, self.H)
        _check(_lib.moeq_router_upload(self._h, wr.ctypes.data, SCORE[score], _stream_ptr(stream)),
               "moeq_router_upload")

    def router(self, x, want_logits=False, stream=None):
        """(topk_ids int32 [T][k], topk_w float32 [T][k], logits float32 [T][E] or None), cuda tensors."""
        import torch
        assert x.is_cuda and x.is_contiguous()
        T = x.shape[0]
        ids = torch.empty((T, self.k), dtype=torch.int32, device=x.device)
        w = torch.empty((T, self.k), dtype=torch.float32, device=x.device)
        z = torch.empty((T, self.E), dtype=torch.float32, device=x.device) if want_logits else None
        _check(_lib.moeq_router(self._h, C.c_void_p(x.data_ptr()), T, C.c_void_p(ids.data_ptr()),
                                C.c_void_p(w.data_ptr()), C.c_void_p(z.data_ptr() if z is not None else 0),
                                _stream_ptr(stream)), "moeq_router")
        return ids, w, z

    def forward_routed(self, x, out=None, stream=None):
        """Router + forward: (out [T][H], topk_ids [T][k], topk_w [T][k]), cuda tensors."""
        import torch
        assert x.is_cuda and x.is_contiguous()
        T = x.shape[0]
        ids = torch.empty((T, self.k), dtype=torch.int32, device=x.device)
        w = torch.empty((T, self.k), dtype=torch.float32, device=x.device)
        if out is None:
            out = torch.empty_like(x)
        _check(_lib.moeq_forward_routed(self._h, C.c_void_p(x.data_ptr()), T, C.c_void_p(ids.data_ptr()),
                                        C.c_void_p(w.data_ptr()), C.c_void_p(out.data_ptr()), _stream_ptr(stream)),
               "moeq_forward_routed")
        return out, ids, w

    def kernel_launches(self) -> int:
        return int(_lib.moeq_kernel_launches(self._h))

    def status(self, clear=False) -> int:
        return int(_lib.moeq_layer_status(self._h, 1 if clear else 0))
