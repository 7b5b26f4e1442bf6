"""Python binding of libna2d.so (include/na2d.h), through ctypes.

Argument marshalling only: every step of the operator runs in the
library's CUDA kernels.  PyTorch supplies device memory and the current
stream.  If the shared library is missing the import of this module
succeeds but every call raises -- there is no other implementation.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading
from typing import NamedTuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libna2d.so")

NA_OK, NA_ERR_INVALID_ARG, NA_ERR_UNSUPPORTED, NA_ERR_CUDA, NA_ERR_DEVICE_TIMEOUT = range(5)
NA_F32, NA_F16, NA_BF16 = 0, 1, 2
_DT = {torch.float32: NA_F32, torch.float16: NA_F16, torch.bfloat16: NA_BF16}

# Every exported symbol of include/na2d.h.
EXPORTS = (
    "na2d_qk_rpb", "na2d_softmax", "na2d_av", "na2d_forward",
    "na2d_forward_host_workspace_bytes", "na2d_forward_host", "na2d_forward_host_noalloc", "na2d_forward_kernel",
    "na2d_device_status", "na2d_debug_timeout_probe", "na_status_str",
    "na2d_backward_workspace_bytes", "na2d_backward", "na2d_sasa_workspace_bytes", "na2d_sasa_forward",
    "na2d_block_workspace_bytes", "na2d_block_forward", "na_forward_nd",
    "na_packed_workspace_bytes", "na_packed_forward", "na_packed_backward_workspace_bytes", "na_packed_backward",
    "na_norm_forward", "na_norm_backward_workspace_bytes", "na_norm_backward",
    "na2d_layer_workspace_bytes", "na2d_layer_forward",
)


class NA2DError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_str(status)}")


_lock = threading.Lock()
_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError(
                f"{path} is missing: build it with `python -m vision_sliding_window_b200.build`"
            )
        lib = ctypes.CDLL(path)
        vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        shape = [i] * 6
        lib.na2d_qk_rpb.argtypes = [vp, vp, vp, vp, *shape, i, vp]
        lib.na2d_softmax.argtypes = [vp, i, i, i, i, i, f, vp]
        lib.na2d_av.argtypes = [vp, vp, vp, *shape, i, vp]
        lib.na2d_forward.argtypes = [vp, vp, vp, vp, vp, *shape, i, vp]
        lib.na2d_forward_host_workspace_bytes.argtypes = [*shape, i]
        lib.na2d_forward_host_workspace_bytes.restype = sz
        lib.na2d_forward_host.argtypes = [vp, vp, vp, vp, vp, vp, sz, *shape, i, vp]
        lib.na2d_forward_host_noalloc.argtypes = [vp, vp, vp, vp, vp, *shape, i, vp]
        lib.na2d_forward_kernel.argtypes = [*shape, i]
        lib.na2d_backward_workspace_bytes.argtypes = [*shape, i]
        lib.na2d_backward_workspace_bytes.restype = sz
        lib.na2d_backward.argtypes = [vp] * 10 + [sz, *shape, i, vp]
        lib.na2d_sasa_workspace_bytes.argtypes = [*shape, i]
        lib.na2d_sasa_workspace_bytes.restype = sz
        lib.na2d_sasa_forward.argtypes = [vp] * 6 + [sz, *shape, i, vp]
        lib.na2d_block_workspace_bytes.argtypes = [*shape, i]
        lib.na2d_block_workspace_bytes.restype = sz
        lib.na2d_block_forward.argtypes = [vp] * 8 + [sz, *shape, i, vp]
        lib.na_forward_nd.argtypes = [vp] * 5 + [i] * 12 + [i, vp]
        ll = ctypes.c_longlong
        packed = [i] * 6
        lib.na_packed_workspace_bytes.argtypes = [*packed, i]
        lib.na_packed_workspace_bytes.restype = sz
        lib.na_packed_forward.argtypes = [vp] * 9 + [sz, *packed, i, i, f, i, vp]
        lib.na_packed_backward_workspace_bytes.argtypes = [*packed, i]
        lib.na_packed_backward_workspace_bytes.restype = sz
        lib.na_packed_backward.argtypes = [vp] * 12 + [sz, *packed, i, i, f, i, vp]
        norm = [ll, i, ll, i, i, f, f, i, vp]
        lib.na_norm_forward.argtypes = [vp] * 9 + norm
        lib.na_norm_backward_workspace_bytes.argtypes = [ll, i, ll, i]
        lib.na_norm_backward_workspace_bytes.restype = sz
        lib.na_norm_backward.argtypes = [vp] * 16 + [sz] + norm
        lib.na2d_layer_workspace_bytes.argtypes = [*shape, i]
        lib.na2d_layer_workspace_bytes.restype = sz
        lib.na2d_layer_forward.argtypes = [vp] * 13 + [sz, *shape, i, i, i, f, f, i, vp]
        lib.na2d_device_status.argtypes = [vp]
        lib.na2d_debug_timeout_probe.argtypes = [ctypes.c_uint, vp]
        lib.na_status_str.argtypes = [i]
        lib.na_status_str.restype = ctypes.c_char_p
        for name in ("na2d_qk_rpb", "na2d_softmax", "na2d_av", "na2d_forward",
                     "na2d_forward_host", "na2d_forward_host_noalloc", "na2d_forward_kernel", "na2d_device_status",
                     "na2d_debug_timeout_probe", "na2d_backward", "na2d_sasa_forward", "na2d_block_forward",
                     "na_forward_nd", "na_packed_forward", "na_packed_backward", "na_norm_forward",
                     "na_norm_backward", "na2d_layer_forward"):
            getattr(lib, name).restype = i
        _lib = lib
        return lib


def status_str(status: int) -> str:
    return load_library().na_status_str(status).decode()


def _check(status: int, what: str):
    if status != NA_OK:
        raise NA2DError(status, what)


def _stream(t: torch.Tensor | None = None):
    dev = t.device if t is not None else torch.device("cuda")
    return ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _need(t: torch.Tensor, name: str, dtype=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")


def _dims(q: torch.Tensor):
    if q.dim() != 5:
        raise ValueError("q/k/v must be [B, heads, H, W, d]")
    return tuple(int(x) for x in q.shape)


def forward(q, k, v, rpb, ksize: int, out=None):
    """Fused NA forward (na2d_forward): returns out [B, heads, H, W, d]."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, q.dtype)
    if rpb is not None:
        _need(rpb, "rpb", q.dtype)
    B, heads, H, W, d = _dims(q)
    out = torch.empty_like(q) if out is None else out
    _need(out, "out", q.dtype)
    _check(load_library().na2d_forward(_ptr(q), _ptr(k), _ptr(v), _ptr(rpb), _ptr(out),
                                       B, heads, H, W, d, ksize, _DT[q.dtype], _stream(q)),
           "na2d_forward")
    return out


def qk_rpb(q, k, rpb, ksize: int, attn=None):
    """Unscaled Eq. (2) logits (na2d_qk_rpb): float32 [B, heads, H, W, ksize^2]."""
    _need(q, "q")
    _need(k, "k", q.dtype)
    if rpb is not None:
        _need(rpb, "rpb", q.dtype)
    B, heads, H, W, d = _dims(q)
    if attn is None:
        attn = torch.empty((B, heads, H, W, ksize * ksize), device=q.device, dtype=torch.float32)
    _need(attn, "attn", torch.float32)
    _check(load_library().na2d_qk_rpb(_ptr(q), _ptr(k), _ptr(rpb), _ptr(attn), B, heads, H, W, d,
                                      ksize, _DT[q.dtype], _stream(q)), "na2d_qk_rpb")
    return attn


def softmax_(attn, ksize: int, scale: float):
    """In-place softmax(scale * attn) over the last axis (na2d_softmax)."""
    _need(attn, "attn", torch.float32)
    B, heads, H, W, kk = (int(x) for x in attn.shape)
    if kk != ksize * ksize:
        raise ValueError("attn last axis must be ksize^2")
    _check(load_library().na2d_softmax(_ptr(attn), B, heads, H, W, ksize, float(scale),
                                       _stream(attn)), "na2d_softmax")
    return attn


def av(attn, v, ksize: int, out=None):
    """Eqs. (3)-(4) with given weights (na2d_av): out [B, heads, H, W, d]."""
    _need(attn, "attn", torch.float32)
    _need(v, "v")
    B, heads, H, W, d = _dims(v)
    out = torch.empty_like(v) if out is None else out
    _need(out, "out", v.dtype)
    _check(load_library().na2d_av(_ptr(attn), _ptr(v), _ptr(out), B, heads, H, W, d, ksize,
                                  _DT[v.dtype], _stream(v)), "na2d_av")
    return out


def backward(q, k, v, rpb, dout, ksize: int, with_rpb_grad: bool = True, workspace=None):
    """Gradients of a scalar loss through the NA forward (na2d_backward):
    returns (dq, dk, dv, drpb), drpb float32 [heads, 2k-1, 2k-1] or None."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (dout, "dout")):
        _need(t, n, q.dtype)
    if rpb is not None:
        _need(rpb, "rpb", q.dtype)
    B, heads, H, W, d = _dims(q)
    lib = load_library()
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    drpb = (torch.empty((heads, 2 * ksize - 1, 2 * ksize - 1), device=q.device, dtype=torch.float32)
            if with_rpb_grad else None)
    need = int(lib.na2d_backward_workspace_bytes(B, heads, H, W, d, ksize, _DT[q.dtype]))
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    _need(workspace, "workspace")
    _check(lib.na2d_backward(_ptr(q), _ptr(k), _ptr(v), _ptr(rpb), _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv),
                             _ptr(drpb), _ptr(workspace), workspace.numel() * workspace.element_size(),
                             B, heads, H, W, d, ksize, _DT[q.dtype], _stream(q)), "na2d_backward")
    return dq, dk, dv, drpb


def sasa_forward(q, k, v, rpb, ksize: int, out=None, workspace=None):
    """SASA, the centred window over a zero-padded map (na2d_sasa_forward):
    returns out [B, heads, H, W, d]."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, q.dtype)
    if rpb is not None:
        _need(rpb, "rpb", q.dtype)
    B, heads, H, W, d = _dims(q)
    out = torch.empty_like(q) if out is None else out
    _need(out, "out", q.dtype)
    lib = load_library()
    need = int(lib.na2d_sasa_workspace_bytes(B, heads, H, W, d, ksize, _DT[q.dtype]))
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    _need(workspace, "workspace")
    _check(lib.na2d_sasa_forward(_ptr(q), _ptr(k), _ptr(v), _ptr(rpb), _ptr(out), _ptr(workspace),
                                 workspace.numel() * workspace.element_size(), B, heads, H, W, d, ksize,
                                 _DT[q.dtype], _stream(q)), "na2d_sasa_forward")
    return out


def block_forward(x, wqkv, bqkv, wo, bo, rpb, heads: int, ksize: int, y=None, workspace=None):
    """An NA block (na2d_block_forward): y = NA(x Wqkv + bqkv) Wo + bo, x and y
    [B, H, W, heads * dh]."""
    for t, n in ((x, "x"), (wqkv, "wqkv"), (wo, "wo")):
        _need(t, n, x.dtype)
    for t, n in ((bqkv, "bqkv"), (bo, "bo"), (rpb, "rpb")):
        if t is not None:
            _need(t, n, x.dtype)
    if x.dim() != 4:
        raise ValueError("x must be [B, H, W, C]")
    B, H, W, C = (int(s) for s in x.shape)
    if C % heads:
        raise ValueError("C must be a multiple of heads")
    dh = C // heads
    y = torch.empty_like(x) if y is None else y
    _need(y, "y", x.dtype)
    lib = load_library()
    need = int(lib.na2d_block_workspace_bytes(B, H, W, heads, dh, ksize, _DT[x.dtype]))
    if need == 0:
        raise NA2DError(NA_ERR_INVALID_ARG, "na2d_block_forward")
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    _need(workspace, "workspace")
    _check(lib.na2d_block_forward(_ptr(x), _ptr(wqkv), _ptr(bqkv), _ptr(wo), _ptr(bo), _ptr(rpb), _ptr(y),
                                  _ptr(workspace), workspace.numel() * workspace.element_size(), B, H, W, heads, dh,
                                  ksize, _DT[x.dtype], _stream(x)), "na2d_block_forward")
    return y


def forward_nd(q, k, v, rpb, ks, dilation=None, out=None):
    """NA over the 1-3 spatial axes of q [B, heads, *spatial, d] with per-axis
    kernel sizes ks and dilations (na_forward_nd)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, n, q.dtype)
    if rpb is not None:
        _need(rpb, "rpb", q.dtype)
    nsp = q.dim() - 3
    if nsp not in (1, 2, 3):
        raise ValueError("q must be [B, heads, *spatial, d] with 1-3 spatial axes")
    ks = tuple(ks) if hasattr(ks, "__len__") else (ks,) * nsp
    dilation = tuple(dilation) if dilation is not None else (1,) * nsp
    B, heads, d = int(q.shape[0]), int(q.shape[1]), int(q.shape[-1])
    L = (1,) * (3 - nsp) + tuple(int(x) for x in q.shape[2:-1])
    kk = (1,) * (3 - nsp) + ks
    dl = (1,) * (3 - nsp) + dilation
    out = torch.empty_like(q) if out is None else out
    _need(out, "out", q.dtype)
    _check(load_library().na_forward_nd(_ptr(q), _ptr(k), _ptr(v), _ptr(rpb), _ptr(out), B, heads, *L, d, *kk, *dl,
                                        _DT[q.dtype], _stream(q)), "na_forward_nd")
    return out


def _need_all(like, dtype, **tensors):
    """_need for every tensor that is given, and that it lies on the device of `like`."""
    where = like.get_device()
    for name, t in tensors.items():
        if t is not None and not (t.get_device() == where and (dtype is None or t.dtype is dtype)
                                  and t.is_contiguous()):
            _need(t, name, dtype)
            raise ValueError(f"{name} is on {t.device}, not on {like.device}")


def _need_shape(t, name, shape):
    if t is not None and t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")


def _workspace(given, need: int, like):
    """The caller's workspace, or one from torch's allocator (None where none is needed)."""
    if given is None:
        return (torch.empty(need, dtype=torch.uint8, device=like.device), need) if need else (None, 0)
    _need_all(like, None, workspace=given)
    return given, given.numel() * given.element_size()


def _enqueue(like, name, tensors, *numbers):
    """Calls the library with the tensors' addresses (None: NULL) and the numbers, on the device of `like` and the
    current stream there."""
    where = like.get_device()
    call = getattr(_lib or load_library(), name)
    at = [None if t is None else t.data_ptr() for t in tensors]
    if where == torch.cuda.current_device():
        status = call(*at, *numbers, _raw_stream(where))
    else:
        with torch.cuda.device(where):
            status = call(*at, *numbers, _raw_stream(where))
    if status != NA_OK:
        raise NA2DError(status, name)


_INT_MAX = 2 ** 31 - 1  # ctypes cuts longer numbers without a word


def _sizes_fit(name, sizes):
    if max(sizes) > _INT_MAX:
        raise NA2DError(NA_ERR_UNSUPPORTED, name)


def _window(n) -> int:
    """A window of more keys than there can be sees as many; a negative one stays so."""
    return max(min(int(n), _INT_MAX), -1)


def _raw_stream(device: int) -> int:
    return torch.cuda.current_stream(device).cuda_stream


if hasattr(torch._C, "_cuda_getCurrentRawStream"):  # the same without building a Stream object
    _raw_stream = torch._C._cuda_getCurrentRawStream


@functools.lru_cache(maxsize=4096)
def _bytes_for(name, *sizes) -> int:
    """A workspace size, which depends on the sizes alone."""
    return int(getattr(load_library(), name)(*sizes))


def _alike(t, where, dtype, shape) -> bool:
    """What _need_all and _need_shape ask of one tensor, without words."""
    return t.get_device() == where and t.dtype is dtype and t.shape == shape and t.is_contiguous()


def _packed_dims(q, k, v, cu_q, cu_k, len_k):
    where, dtype = q.get_device(), q.dtype
    if (where >= 0 and dtype in _DT and q.dim() == 3 and k.dim() == 3 and cu_q.dim() == 1 and cu_q.numel() > 0
            and q.is_contiguous() and k.shape[2] == q.shape[2]):
        ends, i32 = cu_q.shape, torch.int32
        if (_alike(k, where, dtype, k.shape) and _alike(v, where, dtype, k.shape) and _alike(cu_q, where, i32, ends)
                and _alike(cu_k, where, i32, ends) and (len_k is None or _alike(len_k, where, i32, (ends[0] - 1,)))):
            total_q, heads_q, d = q.shape
            total_k, heads_k, _ = k.shape
            return ends[0] - 1, total_q, total_k, heads_q, heads_k, d
    # something is wrong: say what
    _need(q, "q")
    if q.dtype not in _DT:
        raise ValueError(f"q must be float32, float16 or bfloat16, got {q.dtype}")
    _need_all(q, q.dtype, k=k, v=v)
    _need_all(q, torch.int32, cu_q=cu_q, cu_k=cu_k, len_k=len_k)
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q, k and v must be [tokens, heads, d]")
    _need_shape(v, "v", k.shape)
    if cu_q.dim() != 1 or cu_q.numel() < 1:
        raise ValueError("cu_q must be [nseq + 1]")
    _need_shape(cu_k, "cu_k", cu_q.shape)
    _need_shape(len_k, "len_k", (cu_q.numel() - 1,))
    raise ValueError(f"k and v must have q's head size {q.shape[2]}, got {k.shape[2]}")


def packed_forward(q, k, v, cu_q, cu_k, len_k=None, causal: bool = False, window: int = 0, scale=None, out=None,
                   lse=None, workspace=None):
    """Attention over packed sequences (na_packed_forward): returns out
    [total_q, heads_q, d] and lse, float32 [heads_q, total_q].

    q [total_q, heads_q, d]; k, v [total_k, heads_k, d]; sequence s owns the
    rows cu_q[s]:cu_q[s+1] and the key slots cu_k[s]:cu_k[s+1] (int32, on the
    device), of which len_k[s] are filled (None: all).  Causal rows stand at
    the end of their keys and see the last `window` of them (0: all).  scale
    defaults to d ** -0.5.  Rows of no sequence are not written: what a tensor
    that this call allocates holds there is not defined."""
    dims = _packed_dims(q, k, v, cu_q, cu_k, len_k)
    _sizes_fit("na_packed_forward", dims)
    nseq, tq, _, hq, _, d = dims
    if out is None:
        out = torch.empty_like(q)
    else:
        _need_all(q, q.dtype, out=out)
        _need_shape(out, "out", q.shape)
    if lse is None:
        lse = torch.empty((hq, tq), device=q.device, dtype=torch.float32)
    else:
        _need_all(q, torch.float32, lse=lse)
        _need_shape(lse, "lse", (hq, tq))
    dt = _DT[q.dtype]
    need = _bytes_for("na_packed_workspace_bytes", *dims, dt)
    size = 0
    if need or workspace is not None:
        workspace, size = _workspace(workspace, need, q)
    _enqueue(q, "na_packed_forward", (q, k, v, cu_q, cu_k, len_k, out, lse, workspace), size, *dims, int(causal),
             _window(window), d ** -0.5 if scale is None else float(scale), dt)
    return out, lse


def packed_backward(q, k, v, out, lse, dout, cu_q, cu_k, causal: bool = False, window: int = 0, scale=None,
                    grads=None, workspace=None):
    """Gradients through packed_forward (na_packed_backward): returns (dq, dk,
    dv), written into `grads` where given.  out and lse are the forward's;
    rows of no sequence are not written."""
    dims = _packed_dims(q, k, v, cu_q, cu_k, None)
    _sizes_fit("na_packed_backward", dims)
    nseq, tq, _, hq, _, d = dims
    _need_all(q, q.dtype, out=out, dout=dout)
    _need_all(q, torch.float32, lse=lse)
    _need_shape(out, "out", q.shape)
    _need_shape(dout, "dout", q.shape)
    _need_shape(lse, "lse", (hq, tq))
    dq, dk, dv = (torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)) if grads is None else grads
    _need_all(q, q.dtype, dq=dq, dk=dk, dv=dv)
    _need_shape(dq, "dq", q.shape)
    _need_shape(dk, "dk", k.shape)
    _need_shape(dv, "dv", v.shape)
    dt = _DT[q.dtype]
    workspace, size = _workspace(workspace, _bytes_for("na_packed_backward_workspace_bytes", *dims, dt), q)
    _enqueue(q, "na_packed_backward", (q, k, v, out, lse, dout, cu_q, cu_k, dq, dk, dv, workspace), size, *dims,
             int(causal), _window(window), d ** -0.5 if scale is None else float(scale), dt)
    return dq, dk, dv


def _norm_dims(x, o, post, post_w, post_b, gate, w, b):
    """rows, C and gates of a norm's tensors; x is [..., C]."""
    where, dtype, shape = x.get_device(), x.dtype, x.shape
    if where >= 0 and dtype in _DT and len(shape) > 0 and x.is_contiguous():
        C = shape[-1]
        one = (C,)
        if ((o is None or _alike(o, where, dtype, shape)) and (w is None or _alike(w, where, dtype, one))
                and (b is None or _alike(b, where, dtype, one))
                and (post_w is None or post and _alike(post_w, where, dtype, one))
                and (post_b is None or post and _alike(post_b, where, dtype, one))
                and (o is not None or not post and gate is None)):
            rows = x.numel() // C if C else 0
            if gate is None:
                return rows, C, 0
            if gate.dim() in (1, 2) and gate.shape[-1] == C and _alike(gate, where, dtype, gate.shape):
                return rows, C, gate.numel() // C if C else 0
    # something is wrong: say what
    _need(x, "x")
    if x.dtype not in _DT:
        raise ValueError(f"x must be float32, float16 or bfloat16, got {x.dtype}")
    if x.dim() < 1:
        raise ValueError("x must be [..., C]")
    _need_all(x, x.dtype, o=o, post_w=post_w, post_b=post_b, gate=gate, w=w, b=b)
    C = int(x.shape[-1])
    _need_shape(o, "o", x.shape)
    for t, n in ((post_w, "post_w"), (post_b, "post_b"), (w, "w"), (b, "b")):
        _need_shape(t, n, (C,))
    if o is None and (post or gate is not None):
        raise ValueError("post and gate act on o, which is missing")
    if not post and (post_w is not None or post_b is not None):
        raise ValueError("post_w and post_b need post=True")
    raise ValueError("gate must be [C] or [gates, C]")


def norm_forward(x, w=None, b=None, o=None, post: bool = False, post_w=None, post_b=None, gate=None,
                 scale: float = 1.0, eps: float = 1e-5, rms: bool = False, y=None, h=None, norm: bool = True):
    """The norms around a block with its gate and residual (na_norm_forward):
    returns (y, h), y = x + scale * gate . P(o) and h = N(y) w + b.

    x, o, y, h [..., C]; N a LayerNorm, or an RMS norm with rms=True; P the
    same norm with post_w and post_b if post, else the identity.  gate [C] or
    [gates, C] (each row for an equal share of consecutive rows) or None.
    o=None: y is x itself.  norm=False: only y, and h is None."""
    rows, C, gates = _norm_dims(x, o, post, post_w, post_b, gate, w, b)
    _sizes_fit("na_norm_forward", (C,))
    if not norm and (w is not None or b is not None or h is not None or o is None):
        raise ValueError("norm=False takes o, and neither w, b nor h")
    if o is None and y is not None:
        raise ValueError("without o, y is x: there is none to write")
    for t, name in ((y, "y"), (h, "h")):
        if t is not None:
            _need_all(x, x.dtype, **{name: t})
            _need_shape(t, name, x.shape)
    if o is not None and y is None:
        y = torch.empty_like(x)
    if norm and h is None:
        h = torch.empty_like(x)
    _enqueue(x, "na_norm_forward", (x, o, post_w, post_b, gate, w, b, y, h), rows, C, gates, int(rms), int(post),
             float(eps), float(scale), _DT[x.dtype])
    return (x if o is None else y), h


class NormGrads(NamedTuple):
    """What norm_backward returns; None where the input was not given."""
    dx: torch.Tensor
    do: torch.Tensor | None
    dw: torch.Tensor | None
    db: torch.Tensor | None
    dpost_w: torch.Tensor | None
    dpost_b: torch.Tensor | None
    dgate: torch.Tensor | None


def norm_backward(y, dh, dy=None, w=None, b=None, o=None, post: bool = False, post_w=None, post_b=None, gate=None,
                  scale: float = 1.0, eps: float = 1e-5, rms: bool = False, workspace=None) -> NormGrads:
    """Gradients through norm_forward (na_norm_backward), y its first result and
    dh, dy the gradients of both (None: zero).  dx and do have x's type, the
    others are float32 (dgate of gate's shape), zeros where there are no rows."""
    rows, C, gates = _norm_dims(y, o, post, post_w, post_b, gate, w, b)
    _sizes_fit("na_norm_backward", (C,))
    if dh is None and (dy is None or w is not None or b is not None):
        raise ValueError("dh is missing: give dy instead, without w and b")
    _need_all(y, y.dtype, dh=dh, dy=dy)
    _need_shape(dh, "dh", y.shape)
    _need_shape(dy, "dy", y.shape)

    sums = (w, b, post_w, post_b)
    given = [t is not None for t in sums]
    # one allocation for the gradients of all weights of a channel each, every
    # one aligned as the library wants it
    pad = -(-C // 4) * 4
    rest = iter(torch.empty((sum(given), pad), device=y.device, dtype=torch.float32)[:, :C].unbind() if any(given)
                else ())
    g = NormGrads(torch.empty_like(y), None if o is None else torch.empty_like(y),
                  *(next(rest) if there else None for there in given),
                  None if gate is None else torch.empty(gate.shape, device=y.device, dtype=torch.float32))
    if rows == 0:  # which the library refuses: its kernels would leave the sums unwritten
        for t in g:
            if t is not None:
                t.zero_()
        return g
    dt = _DT[y.dtype]
    workspace, size = _workspace(workspace, _bytes_for("na_norm_backward_workspace_bytes", rows, C, gates, dt), y)
    _enqueue(y, "na_norm_backward", (y, o, post_w, post_b, gate, w, dy, dh, *g, workspace), size, rows, C, gates,
             int(rms), int(post), float(eps), float(scale), dt)
    return g


def layer_forward(x, w, b, wqkv, bqkv, wo, bo, rpb, heads: int, ksize: int, gate=None, post: bool = False,
                  post_w=None, post_b=None, scale: float = 1.0, eps: float = 1e-5, rms: bool = False, y=None,
                  workspace=None):
    """The attention half of a NAT layer (na2d_layer_forward): returns
    x + scale * gate . P(block(N(x) w + b)), x [B, H, W, heads * dh]; the block's
    arguments as in block_forward, the norms' as in norm_forward."""
    if x.dim() != 4:
        raise ValueError("x must be [B, H, W, C]")
    _, C, gates = _norm_dims(x, x, post, post_w, post_b, gate, w, b)
    _need_all(x, x.dtype, wqkv=wqkv, bqkv=bqkv, wo=wo, bo=bo, rpb=rpb)
    if heads < 1 or C % heads:
        raise ValueError("C must be a multiple of heads")
    B, H, W = (int(n) for n in x.shape[:3])
    for t, n, shape in ((wqkv, "wqkv", (C, 3 * C)), (bqkv, "bqkv", (3 * C,)), (wo, "wo", (C, C)), (bo, "bo", (C,)),
                        (rpb, "rpb", (heads, 2 * ksize - 1, 2 * ksize - 1))):
        _need_shape(t, n, shape)
    y = torch.empty_like(x) if y is None else y
    _need_all(x, x.dtype, y=y)
    _need_shape(y, "y", x.shape)
    dt, dims = _DT[x.dtype], (B, H, W, heads, C // heads, ksize)
    _sizes_fit("na2d_layer_forward", (*dims, gates))
    workspace, size = _workspace(workspace, _bytes_for("na2d_layer_workspace_bytes", *dims, dt), x)
    _enqueue(x, "na2d_layer_forward", (x, w, b, wqkv, bqkv, wo, bo, rpb, post_w, post_b, gate, y, workspace), size,
             *dims, gates, int(rms), int(post), float(eps), float(scale), dt)
    return y


def host_workspace_bytes(B, heads, H, W, d, ksize, dtype) -> int:
    return int(load_library().na2d_forward_host_workspace_bytes(B, heads, H, W, d, ksize, _DT[dtype]))


def forward_host(q_host, k_host, v_host, rpb_host, out_host, ksize: int, workspace, stream=None):
    """na2d_forward_host: host tensors in and out, a caller-owned device workspace."""
    B, heads, H, W, d = _dims(q_host)
    for t in (q_host, k_host, v_host, out_host) + ((rpb_host,) if rpb_host is not None else ()):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError("host buffers must be contiguous CPU tensors")
    _need(workspace, "workspace")
    st = ctypes.c_void_p(stream.cuda_stream) if stream is not None else _stream(workspace)
    _check(load_library().na2d_forward_host(
        _ptr(q_host), _ptr(k_host), _ptr(v_host), _ptr(rpb_host), _ptr(out_host), _ptr(workspace),
        workspace.numel() * workspace.element_size(), B, heads, H, W, d, ksize, _DT[q_host.dtype], st),
        "na2d_forward_host")
    return out_host


def forward_host_noalloc(q_host, k_host, v_host, rpb_host, out_host, ksize: int, stream=None):
    """na2d_forward_host_noalloc: host tensors in and out, staged in the
    library's own fixed device array, for callers that cannot allocate device
    memory; shapes needing more than NOALLOC_SCRATCH_BYTES are rejected."""
    B, heads, H, W, d = _dims(q_host)
    for t in (q_host, k_host, v_host, out_host) + ((rpb_host,) if rpb_host is not None else ()):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError("host buffers must be contiguous CPU tensors")
    st = ctypes.c_void_p(stream.cuda_stream) if stream is not None else _stream()
    _check(load_library().na2d_forward_host_noalloc(
        _ptr(q_host), _ptr(k_host), _ptr(v_host), _ptr(rpb_host), _ptr(out_host), B, heads, H, W, d, ksize,
        _DT[q_host.dtype], st), "na2d_forward_host_noalloc")
    return out_host


NOALLOC_SCRATCH_BYTES = 64 << 20  # NA2D_NOALLOC_SCRATCH_BYTES of include/na2d.h


def forward_kernel(B, heads, H, W, d, ksize, dtype) -> int:
    """1 if na2d_forward runs the tensor-core kernel for these arguments, 0 for SIMT."""
    return int(load_library().na2d_forward_kernel(B, heads, H, W, d, ksize, _DT[dtype]))


def device_status(stream=None) -> int:
    st = ctypes.c_void_p(stream.cuda_stream) if stream is not None else _stream()
    return int(load_library().na2d_device_status(st))


def debug_timeout_probe(timeout_us: int, stream=None) -> int:
    st = ctypes.c_void_p(stream.cuda_stream) if stream is not None else _stream()
    return int(load_library().na2d_debug_timeout_probe(int(timeout_us), st))
