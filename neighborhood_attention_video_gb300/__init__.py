"""Python binding of the GB300 NA3D forward library (``libna3d.so``).

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI declared in ``include/na3d.h``. There is no CPU or
PyTorch fallback; if the library has not been built, importing works but any
call raises ``NA3DUnavailable``.

PyTorch is used for device memory and streams only.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

__all__ = [
    "NA3DError", "NA3DUnavailable", "na3d_attention", "na3d_fwd", "na3d_fwd_strided", "na3d_fwd_region",
    "na3d_qkv_proj", "qkv_views", "na3d_scored_fwd", "na3d_scored_attention", "na3d_scored_bwd",
    "na3d_lora_qkv_proj", "na3d_lora_qkv_proj_bwd", "na3d_lora_workspace",
    "na3d_rope_table", "na3d_norm_rope", "na3d_norm_rope_bwd", "na3d_norm_rope_workspace",
    "na3d_cross_fwd", "na3d_cross_attention", "na3d_cross_bwd", "na3d_cross_workspace",
    "na3d_scored_bwd_workspace", "na3d_status_string", "na3d_plan",
    "na3d_device_status", "library_path", "load_library", "EXPORTED_SYMBOLS",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libna3d.so")
EXPORTED_SYMBOLS = ("na3d_fwd", "na3d_fwd_strided", "na3d_fwd_region", "na3d_qkv_proj",
                    "na3d_scored_fwd", "na3d_scored_bwd", "na3d_scored_bwd_workspace",
                    "na3d_lora_qkv_proj", "na3d_lora_qkv_proj_bwd", "na3d_lora_workspace",
                    "na3d_rope_table", "na3d_norm_rope", "na3d_norm_rope_bwd", "na3d_norm_rope_workspace",
                    "na3d_cross_fwd", "na3d_cross_bwd", "na3d_cross_workspace",
                    "na3d_selftest_withhold", "na3d_cross_selftest_withhold", "na3d_status_string", "na3d_plan",
                    "na3d_device_status")

NA3D_OK = 0
_I64 = ctypes.c_int64
_P = ctypes.c_void_p
_F32 = ctypes.c_float
_F64 = ctypes.c_double
_lib = None


class NA3DError(RuntimeError):
    """A non-zero status returned by the C ABI."""

    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {na3d_status_string(status)} (status {status})")


class NA3DUnavailable(RuntimeError):
    """The CUDA library is missing: build it with ``__graft_entry__.build()``."""


class PlanInfo(ctypes.Structure):
    _fields_ = [("bt", ctypes.c_int32), ("bh", ctypes.c_int32), ("bw", ctypes.c_int32),
                ("cw", ctypes.c_int32), ("cr", ctypes.c_int32), ("n_mma", ctypes.c_int32),
                ("hd_box", ctypes.c_int32), ("stages", ctypes.c_int32),
                ("bricks_per_slice", ctypes.c_int64), ("chunks_per_slice", ctypes.c_int64),
                ("smem_bytes", ctypes.c_int64), ("w_stride", ctypes.c_int32),
                ("tile_cap", ctypes.c_int32)]


def library_path() -> str:
    return LIB_PATH


def load_library():
    """Load ``libna3d.so`` (once) and declare the C signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise NA3DUnavailable(
            f"{LIB_PATH} is missing; build it with `python -c 'import __graft_entry__ as g; g.build()'`")
    lib = ctypes.CDLL(LIB_PATH)
    lib.na3d_fwd.argtypes = [_P, _P, _P, _P] + [_I64] * 9 + [_P]
    lib.na3d_fwd.restype = ctypes.c_int
    lib.na3d_fwd_strided.argtypes = [_P, _P, _P, _P] + [_I64] * 12 + [_P]
    lib.na3d_fwd_strided.restype = ctypes.c_int
    lib.na3d_fwd_region.argtypes = [_P, _P, _P, _P] + [_I64] * 18 + [_P]
    lib.na3d_fwd_region.restype = ctypes.c_int
    lib.na3d_qkv_proj.argtypes = [_P, _P, _P, _P] + [_I64] * 4 + [_P]
    lib.na3d_qkv_proj.restype = ctypes.c_int
    lib.na3d_scored_fwd.argtypes = [_P] * 5 + [_I64] * 12 + [_F32] + [_P] * 4
    lib.na3d_scored_fwd.restype = ctypes.c_int
    lib.na3d_scored_bwd.argtypes = [_P] * 10 + [_I64] * 15 + [_F32] + [_P] * 4
    lib.na3d_scored_bwd.restype = ctypes.c_int
    lib.na3d_scored_bwd_workspace.argtypes = [_I64] * 5
    lib.na3d_scored_bwd_workspace.restype = _I64
    lib.na3d_lora_qkv_proj.argtypes = [_P] * 10 + [_I64] * 7 + [_P]
    lib.na3d_lora_qkv_proj.restype = ctypes.c_int
    lib.na3d_lora_qkv_proj_bwd.argtypes = [_P] * 12 + [_I64] * 7 + [_P]
    lib.na3d_lora_qkv_proj_bwd.restype = ctypes.c_int
    lib.na3d_lora_workspace.argtypes = [_I64] * 7 + [ctypes.c_int]
    lib.na3d_lora_workspace.restype = _I64
    lib.na3d_rope_table.argtypes = [_P] + [_I64] * 6 + [_F64] * 7 + [_P]
    lib.na3d_rope_table.restype = ctypes.c_int
    rope_how = [ctypes.c_int, _F32, _F32, _F32, ctypes.c_int, _P]
    lib.na3d_norm_rope.argtypes = [_P] * 7 + [_I64] * 14 + rope_how
    lib.na3d_norm_rope.restype = ctypes.c_int
    lib.na3d_norm_rope_bwd.argtypes = [_P] * 12 + [_I64] * 16 + rope_how
    lib.na3d_norm_rope_bwd.restype = ctypes.c_int
    lib.na3d_norm_rope_workspace.argtypes = [_I64]
    lib.na3d_norm_rope_workspace.restype = _I64
    lib.na3d_cross_fwd.argtypes = [_P] * 6 + [_I64] * 9 + [_P] * 3
    lib.na3d_cross_fwd.restype = ctypes.c_int
    lib.na3d_cross_bwd.argtypes = [_P] * 10 + [_I64] * 12 + [_P] * 3
    lib.na3d_cross_bwd.restype = ctypes.c_int
    lib.na3d_cross_workspace.argtypes = [_I64] * 6 + [ctypes.c_int]
    lib.na3d_cross_workspace.restype = _I64
    lib.na3d_selftest_withhold.argtypes = [_P, _P, _P, _P] + [_I64] * 10 + [_P]
    lib.na3d_selftest_withhold.restype = ctypes.c_int
    lib.na3d_cross_selftest_withhold.argtypes = [_P] * 10 + [_I64] * 6 + [_P] * 3
    lib.na3d_cross_selftest_withhold.restype = ctypes.c_int
    lib.na3d_status_string.argtypes = [ctypes.c_int]
    lib.na3d_status_string.restype = ctypes.c_char_p
    lib.na3d_plan.argtypes = [_I64] * 8 + [ctypes.POINTER(PlanInfo)]
    lib.na3d_plan.restype = ctypes.c_int
    lib.na3d_device_status.argtypes = [_P]
    lib.na3d_device_status.restype = ctypes.c_int
    _lib = lib
    return lib


def na3d_status_string(status: int) -> str:
    return load_library().na3d_status_string(int(status)).decode()


_torch = None
_cuda_ok = None   # torch.cuda.is_available(), fixed for the process
_get_device = None


def _torch_module():
    global _torch, _cuda_ok, _get_device
    if _torch is None:
        import torch
        ok = torch.cuda.is_available()
        if ok:
            torch.cuda.init()   # which torch.cuda.current_device() does, and the call that is quicker does not
            _get_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
        _torch, _cuda_ok = torch, ok
    return _torch


def _device() -> int:
    """The current CUDA device, -2 where there is none (behind _torch_module())."""
    return _get_device() if _cuda_ok else -2


def _check_bf16_on_device(tensors):
    """Each (name, tensor) is a bf16 tensor on the current CUDA device: the
    kernels get raw pointers, so a host or other-device tensor must not pass."""
    torch = _torch_module()
    dev = _device()
    for name, t in tensors:
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dtype is not torch.bfloat16 or t.get_device() != dev:
            raise TypeError(f"{name} must be a bfloat16 tensor on the current CUDA device")


def _stream_handle(stream) -> int:
    if stream is None:   # the current torch stream of the current device
        torch = _torch_module()
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None:
            return raw(_device() if _cuda_ok else torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def na3d_fwd(q, k, v, out, kernel_size, stream=None) -> None:
    """out = NA3D(q, k, v) for bf16 CUDA tensors of shape (B, T, H, W, NH, HD).

    ``q`` must already be scaled by HD**-0.5. ``kernel_size`` = (KT, KH, KW),
    odd. ``out`` is written in place. Runs asynchronously on ``stream``
    (default: the current torch stream). Raises NA3DError on a bad argument.
    """
    lib = _lib if _lib is not None else load_library()
    _check_bf16_on_device((("q", q), ("k", k), ("v", v), ("out", out)))
    shape = q.shape
    if len(shape) != 6 or k.shape != shape or v.shape != shape or out.shape != shape:
        raise ValueError("q, k, v and out must have the same 6-D (B,T,H,W,NH,HD) shape")
    if not (q.is_contiguous() and k.is_contiguous() and v.is_contiguous() and out.is_contiguous()):
        raise ValueError("q, k, v and out must be contiguous")
    KT, KH, KW = (int(x) for x in kernel_size)
    rc = lib.na3d_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                      *shape, KT, KH, KW, _stream_handle(stream))
    if rc != NA3D_OK:
        raise NA3DError(rc, "na3d_fwd")


def na3d_attention(q, k, v, kernel_size, stream=None):
    """Returns a new tensor out = NA3D(q, k, v): ``na3d_fwd`` with the output
    allocated like ``q`` (contiguous bf16 (B, T, H, W, NH, HD) on its device).
    q must already be scaled by HD**-0.5."""
    torch = _torch_module()
    out = torch.empty_like(q, memory_format=torch.contiguous_format)
    na3d_fwd(q, k, v, out, kernel_size, stream=stream)
    return out


def _token_stride(name, t) -> int:
    """Elements between consecutive (b,t,h,w) positions of a (B,T,H,W,NH,HD)
    view whose heads are packed (head stride HD, unit element stride)."""
    st, sh = t.stride(), t.shape
    if (st[5] == 1 and st[4] == sh[5] and st[2] == sh[3] * st[3] and st[1] == sh[2] * st[2]
            and st[0] == sh[1] * st[1]):
        return st[3]
    if st[5] != 1 or (sh[4] > 1 and st[4] != sh[5]):
        raise ValueError(f"{name}: heads must be packed (strides [..., HD, 1])")
    step = span = None   # axes of one position say nothing about the step
    for i in (3, 2, 1, 0):
        if sh[i] == 1:
            continue
        if step is None:
            step = st[i]
        elif st[i] != span:
            raise ValueError(f"{name}: grid positions must share one token stride")
        span = sh[i] * st[i]
    return int(sh[4] * sh[5] if step is None else step)


def na3d_fwd_strided(q, k, v, out, kernel_size, stream=None) -> None:
    """``na3d_fwd`` for q, k, v views with a token stride, e.g. the three
    slices ``x[..., 0, :, :]``, ``x[..., 1, :, :]``, ``x[..., 2, :, :]`` of a
    fused projection output ``x`` of shape (B, T, H, W, 3, NH, HD). ``out`` is
    a contiguous (B, T, H, W, NH, HD) bf16 CUDA tensor."""
    lib = load_library()
    _check_bf16_on_device((("q", q), ("k", k), ("v", v), ("out", out)))
    for t in (q, k, v, out):
        if t.dim() != 6 or tuple(t.shape) != tuple(q.shape):
            raise ValueError("q, k, v and out must have the same 6-D shape")
    if not out.is_contiguous():
        raise ValueError("out must be contiguous")
    strides = [_token_stride(n, t) for n, t in (("q", q), ("k", k), ("v", v))]
    KT, KH, KW = (int(x) for x in kernel_size)
    rc = lib.na3d_fwd_strided(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                              *[int(x) for x in q.shape], KT, KH, KW, *strides,
                              _stream_handle(stream))
    if rc != NA3D_OK:
        raise NA3DError(rc, "na3d_fwd_strided")


def na3d_fwd_region(q, k, v, out, kernel_size, offset, stream=None) -> None:
    """``out`` = the rows of NA3D on the whole grid at the query box
    ``offset`` = (t0, h0, w0) with the extents of ``q``: q and out have shape
    (B, Tq, Hq, Wq, NH, HD), k and v (B, T, H, W, NH, HD). Every query keeps
    its window in the whole grid (global coordinates). q, k, v may be views
    with a token stride as in ``na3d_fwd_strided``; ``out`` is contiguous."""
    lib = load_library()
    _check_bf16_on_device((("q", q), ("k", k), ("v", v), ("out", out)))
    for name, t in (("q", q), ("k", k), ("v", v), ("out", out)):
        if t.dim() != 6:
            raise ValueError(f"{name} must be a 6-D tensor")
    if tuple(k.shape) != tuple(v.shape) or tuple(out.shape) != tuple(q.shape):
        raise ValueError("k and v must share a shape, and so must q and out")
    if q.shape[0] != k.shape[0] or q.shape[4:] != k.shape[4:]:
        raise ValueError("q and k must agree on B, NH and HD")
    if not out.is_contiguous():
        raise ValueError("out must be contiguous")
    strides = [_token_stride(n, t) for n, t in (("q", q), ("k", k), ("v", v))]
    KT, KH, KW = (int(x) for x in kernel_size)
    t0, h0, w0 = (int(x) for x in offset)
    B, T, H, W, NH, HD = (int(x) for x in k.shape)
    Tq, Hq, Wq = (int(x) for x in q.shape[1:4])
    rc = lib.na3d_fwd_region(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                             B, T, H, W, NH, HD, KT, KH, KW, t0, h0, w0, Tq, Hq, Wq,
                             *strides, _stream_handle(stream))
    if rc != NA3D_OK:
        raise NA3DError(rc, "na3d_fwd_region")


def na3d_qkv_proj(x, w, bias, qkv, num_heads, head_dim, stream=None) -> None:
    """qkv = x w^T (+ bias), the q block scaled by head_dim**-0.5 (see
    ``na3d_qkv_proj`` in include/na3d.h). x: contiguous bf16 CUDA tensor
    (..., C); w: (3*NH*HD, C); bias: (3*NH*HD,) or None; qkv: contiguous bf16
    with x's leading dimensions and 3*NH*HD elements per token, e.g.
    (B, T, H, W, 3, NH, HD). ``qkv_views`` gives the attention inputs."""
    lib = load_library()
    tensors = [("x", x), ("w", w), ("qkv", qkv)] + ([("bias", bias)] if bias is not None else [])
    _check_bf16_on_device(tensors)
    for name, t in tensors:
        if not t.is_contiguous():
            raise TypeError(f"{name} must be a contiguous bfloat16 CUDA tensor")
    NH, HD = int(num_heads), int(head_dim)
    C = int(x.shape[-1])
    M = x.numel() // C if C else 0
    N = 3 * NH * HD
    if tuple(w.shape) != (N, C) or (bias is not None and tuple(bias.shape) != (N,)):
        raise ValueError("w must be (3*NH*HD, C) and bias (3*NH*HD,)")
    if qkv.numel() != M * N:
        raise ValueError("qkv must hold 3*NH*HD values per token of x")
    rc = lib.na3d_qkv_proj(x.data_ptr(), w.data_ptr(), bias.data_ptr() if bias is not None else None,
                           qkv.data_ptr(), M, C, NH, HD, _stream_handle(stream))
    if rc != NA3D_OK:
        raise NA3DError(rc, "na3d_qkv_proj")


def qkv_views(qkv):
    """q, k, v views (B, T, H, W, NH, HD) of a (B, T, H, W, 3, NH, HD)
    projection output, for ``na3d_fwd_strided``."""
    if _torch is not None and isinstance(qkv, _torch.Tensor):   # 3 us less than by index
        return qkv.select(-3, 0), qkv.select(-3, 1), qkv.select(-3, 2)
    return qkv[..., 0, :, :], qkv[..., 1, :, :], qkv[..., 2, :, :]


def _check_one(torch, dev, name, t, dtype, shape):
    """t is a contiguous tensor of that dtype and shape on device `dev`."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype or t.get_device() != dev:
        raise TypeError(f"{name} must be a {dtype} tensor on the current CUDA device")
    if t.shape != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}, not {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _check_on_device(tensors):
    """Each (name, tensor, dtype, shape) is a contiguous tensor of that dtype
    and shape on the current CUDA device."""
    torch = _torch_module()
    dev = _device()
    for name, t, dtype, shape in tensors:
        _check_one(torch, dev, name, t, dtype, shape)


def _check_bf16_of_shape(shape, names, tensors):
    """The tensors are bf16, of one 6-D shape, on the current CUDA device."""
    torch = _torch_module()
    dev, bf16 = _device(), torch.bfloat16
    for name, t in zip(names, tensors):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dtype is not bf16 or t.get_device() != dev:
            raise TypeError(f"{name} must be a bfloat16 tensor on the current CUDA device")
        if t.shape != shape:
            raise ValueError(f"{name} must have the (B,T,H,W,NH,HD) shape of q")
    if len(shape) != 6:
        raise ValueError("q must have a 6-D (B,T,H,W,NH,HD) shape")


def _empty_on(stream, device, shape, dtype):
    """A new tensor on `device`, allocated on the stream that the call uses, so
    that the allocator may reuse its memory only behind the call."""
    torch = _torch_module()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _empty(stream, like, shape, dtype):
    """``_empty_on`` the device of `like`."""
    return _empty_on(stream, like.device, shape, dtype)


_kept = threading.local()   # a thread's workspaces, by device and stream; 16 at most


def _workspace(work, need, like, stream):
    """`work` where it is given and large enough. Else a workspace that this
    thread keeps for the current stream: its calls run there one after another
    (a new one for each call took 8 us of a 28 us call). A call on a stream of
    the caller's, or one that is being captured and may be replayed beside later
    calls, gets one of its own."""
    torch = _torch_module()
    if work is None:
        if stream is not None or torch.cuda.is_current_stream_capturing():
            return _empty(stream, like, (need,), torch.uint8)
        kept = _kept.__dict__
        key = (like.get_device(), _stream_handle(None))
        work = kept.get(key)
        if work is None or work.numel() < need:
            if len(kept) >= 16:
                kept.clear()
            work = kept[key] = _empty(None, like, (need,), torch.uint8)
        return work
    dev = _device()
    if not isinstance(work, torch.Tensor) or work.get_device() != dev or not work.is_contiguous():
        raise TypeError("work must be a contiguous tensor on the current CUDA device")
    if work.numel() * work.element_size() < need:
        raise ValueError(f"work must hold {need} bytes")
    return work


def _scored_options(shape, softcap, slopes, doc, prefix):
    """The score arguments of the na3d_scored_ calls, checked: (softcap, the
    three pointers or None)."""
    torch = _torch_module()
    dev = _device()
    ps = pd = pp = None
    if slopes is not None:
        _check_one(torch, dev, "slopes", slopes, torch.float32, (shape[4], 3))
        ps = slopes.data_ptr()
    if doc is not None:
        _check_one(torch, dev, "doc", doc, torch.int32, shape[:4])
        pd = doc.data_ptr()
    if prefix is not None:
        _check_one(torch, dev, "prefix", prefix, torch.int32, shape[:1])
        pp = prefix.data_ptr()
    return softcap, ps, pd, pp


def _token_strides(names, tensors):
    """``_token_stride`` of tensors of one shape, which often share strides."""
    first = tensors[0].stride()
    ts = _token_stride(names[0], tensors[0])
    return [ts if t.stride() == first else _token_stride(n, t) for n, t in zip(names, tensors)]


def _shape_of(q):
    if not isinstance(q, _torch_module().Tensor):
        raise TypeError("q must be a torch.Tensor")
    return q.shape


def _call_scored_fwd(q, k, v, out, lse, shape, kernel_size, softcap, slopes, doc, prefix, stream) -> None:
    """The call behind na3d_scored_fwd: out and lse are as it needs them."""
    lib = _lib if _lib is not None else load_library()
    KT, KH, KW = kernel_size
    rc = lib.na3d_scored_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                             None if lse is None else lse.data_ptr(), *shape, int(KT), int(KH), int(KW),
                             *_token_strides(("q", "k", "v"), (q, k, v)),
                             *_scored_options(shape, softcap, slopes, doc, prefix), _stream_handle(stream))
    if rc != NA3D_OK:
        raise NA3DError(rc, "na3d_scored_fwd")


def na3d_scored_fwd(q, k, v, out, kernel_size, lse=None, softcap=0.0, slopes=None, doc=None, prefix=None,
                    stream=None) -> None:
    """``na3d_fwd_strided`` with shaped scores (see ``na3d_scored_fwd`` in
    include/na3d.h): a tanh cap (``softcap`` > 0), a bias that falls with the
    distance (``slopes``: fp32 (NH, 3), per head along T, H and W), a document
    mask (``doc``: int32 (B, T, H, W), negative for padding) and a causal mask
    along T with a free prefix (``prefix``: int32 (B,) frames). ``lse``, where
    given, receives the fp32 (B, T, H, W, NH) log-sum-exp of the scores. q, k,
    v may be views with a token stride; ``out`` is contiguous. HD up to 128.
    Windows are taken on the whole grid and cut by the masks, so a packed clip
    has fewer keys next to a cut than the clip by itself; ``prefix`` counts from
    the entry's first frame. Autograd does not see the call: outputs have no
    graph, the gradients come from ``na3d_scored_bwd``."""
    shape = _shape_of(q)
    _check_bf16_of_shape(shape, ("q", "k", "v", "out"), (q, k, v, out))
    if not out.is_contiguous():
        raise ValueError("out must be contiguous")
    if lse is not None:
        _check_on_device((("lse", lse, _torch.float32, shape[:5]),))
    _call_scored_fwd(q, k, v, out, lse, shape, kernel_size, softcap, slopes, doc, prefix, stream)


def na3d_scored_attention(q, k, v, kernel_size, softcap=0.0, slopes=None, doc=None, prefix=None,
                          return_lse=False, stream=None):
    """``na3d_scored_fwd`` into a new tensor: returns out, or (out, lse) where
    ``return_lse`` is true (what ``na3d_scored_bwd`` needs)."""
    torch = _torch_module()
    shape = _shape_of(q)
    _check_bf16_of_shape(shape, ("q", "k", "v"), (q, k, v))
    out = _empty(stream, q, shape, torch.bfloat16)
    lse = _empty(stream, q, shape[:-1], torch.float32) if return_lse else None
    _call_scored_fwd(q, k, v, out, lse, shape, kernel_size, softcap, slopes, doc, prefix, stream)
    return (out, lse) if return_lse else out


def na3d_scored_bwd_workspace(B, T, H, W, NH) -> int:
    """Bytes of workspace that ``na3d_scored_bwd`` uses."""
    need = int(load_library().na3d_scored_bwd_workspace(B, T, H, W, NH))
    if need < 0:
        raise ValueError("every size must be at least 1")
    return need


def na3d_scored_bwd(q, k, v, out, lse, dout, dq, dk, dv, kernel_size, softcap=0.0, slopes=None, doc=None,
                    prefix=None, work=None, stream=None) -> None:
    """dq, dk, dv = the gradients of ``na3d_scored_fwd`` for the gradient
    ``dout`` of its output. ``out`` and ``lse`` are what the forward pass wrote;
    the other arguments are the forward pass's. dq, dk and dv may be views with
    a token stride, e.g. ``qkv_views`` of a fused gradient. ``work``: a tensor of
    ``na3d_scored_bwd_workspace`` bytes, kept by the caller (one call at a time);
    None takes one that the binding keeps (for this thread and the current
    stream; a call with a ``stream`` or under capture allocates its own)."""
    lib = _lib if _lib is not None else load_library()
    shape = _shape_of(q)
    _check_bf16_of_shape(shape, ("q", "k", "v", "out", "dout", "dq", "dk", "dv"), (q, k, v, out, dout, dq, dk, dv))
    if not (out.is_contiguous() and dout.is_contiguous()):
        raise ValueError("out and dout must be contiguous")
    _check_on_device((("lse", lse, _torch.float32, shape[:5]),))
    options = _scored_options(shape, softcap, slopes, doc, prefix)
    strides = _token_strides(("q", "k", "v", "dq", "dk", "dv"), (q, k, v, dq, dk, dv))
    KT, KH, KW = kernel_size
    work = _workspace(work, lib.na3d_scored_bwd_workspace(*shape[:5]), q, stream)
    rc = lib.na3d_scored_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                             dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), work.data_ptr(),
                             *shape, int(KT), int(KH), int(KW), *strides, *options, _stream_handle(stream))
    if rc != NA3D_OK:
        raise NA3DError(rc, "na3d_scored_bwd")


def na3d_lora_workspace(M, C, num_heads, head_dim, rank, n_requests, n_adapters, backward=False) -> int:
    """Bytes of workspace of ``na3d_lora_qkv_proj``, or of its backward pass."""
    need = int(load_library().na3d_lora_workspace(M, C, num_heads, head_dim, rank, n_requests, n_adapters,
                                                  1 if backward else 0))
    if need < 0:
        raise ValueError("sizes that na3d_lora_qkv_proj does not take")
    return need


def _check_lora(x, w, lora_a, lora_b, scaling, offsets, adapter, num_heads, head_dim):
    """The arguments both directions share, checked: (M, C, NH, HD, R, n_req, n_ad)."""
    torch = _torch_module()
    bf16, i32 = torch.bfloat16, torch.int32
    NH, HD = int(num_heads), int(head_dim)
    for name, t, dims in (("x", x, None), ("lora_a", lora_a, 3), ("adapter", adapter, 1)):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dim() == 0 or (dims and t.dim() != dims):
            raise ValueError(f"{name} has the wrong number of dimensions")
    C, N = int(x.shape[-1]), 3 * NH * HD
    n_ad, R, n_req = int(lora_a.shape[0]), int(lora_a.shape[1]), int(adapter.shape[0])
    _check_on_device((("x", x, bf16, x.shape), ("w", w, bf16, (N, C)), ("lora_a", lora_a, bf16, (n_ad, R, C)),
                      ("lora_b", lora_b, bf16, (n_ad, N, R)), ("scaling", scaling, torch.float32, (n_ad,)),
                      ("offsets", offsets, i32, (n_req + 1,)), ("adapter", adapter, i32, (n_req,))))
    return (x.numel() // C if C else 0), C, NH, HD, R, n_req, n_ad


def na3d_lora_qkv_proj(x, w, bias, lora_a, lora_b, scaling, offsets, adapter, qkv, num_heads, head_dim, work=None,
                       stream=None) -> None:
    """``na3d_qkv_proj`` with a low-rank adapter for each request of the batch
    (see ``na3d_lora_qkv_proj`` in include/na3d.h). Tokens
    offsets[r] .. offsets[r+1] - 1 of x are request r's, with the adapter
    adapter[r] (none where the id is not 0 .. n_adapters - 1): lora_a
    (n_adapters, R, C) and lora_b (n_adapters, 3*NH*HD, R) in bf16, scaling fp32
    (n_adapters,); offsets int32 (n_requests + 1,) and adapter int32
    (n_requests,) on the device. R is a multiple of 8 up to 128. ``work``: a
    tensor of ``na3d_lora_workspace`` bytes, kept by the caller (one call at a
    time); None takes one that the binding keeps (for this thread and the current
    stream; a call with a ``stream`` or under capture allocates its own).
    Autograd does not see the call: the gradients come from
    ``na3d_lora_qkv_proj_bwd``."""
    lib = _lib if _lib is not None else load_library()
    sizes = _check_lora(x, w, lora_a, lora_b, scaling, offsets, adapter, num_heads, head_dim)
    _check_bf16_on_device((("qkv", qkv),))
    if bias is not None:
        _check_on_device((("bias", bias, _torch.bfloat16, w.shape[:1]),))
    if not qkv.is_contiguous():
        raise ValueError("qkv must be contiguous")
    if qkv.numel() != sizes[0] * w.shape[0]:
        raise ValueError("qkv must hold 3*NH*HD values per token of x")
    work = _workspace(work, max(0, lib.na3d_lora_workspace(*sizes, 0)), x, stream)
    rc = lib.na3d_lora_qkv_proj(x.data_ptr(), w.data_ptr(), None if bias is None else bias.data_ptr(),
                                lora_a.data_ptr(), lora_b.data_ptr(), scaling.data_ptr(), offsets.data_ptr(),
                                adapter.data_ptr(), qkv.data_ptr(), work.data_ptr(), *sizes, _stream_handle(stream))
    if rc != NA3D_OK:
        raise NA3DError(rc, "na3d_lora_qkv_proj")


def na3d_lora_qkv_proj_bwd(dqkv, x, w, lora_a, lora_b, scaling, offsets, adapter, dx, dlora_a, dlora_b, num_heads,
                           head_dim, work=None, stream=None) -> None:
    """The gradients of ``na3d_lora_qkv_proj`` with respect to x (``dx``, or
    None where it is not wanted) and the adapters, for the gradient ``dqkv`` of
    its output; the base weight, the bias and the scalings are frozen. ``work``:
    as there, with ``backward=True``."""
    lib = _lib if _lib is not None else load_library()
    sizes = _check_lora(x, w, lora_a, lora_b, scaling, offsets, adapter, num_heads, head_dim)
    bf16 = _torch.bfloat16
    _check_bf16_on_device((("dqkv", dqkv),))
    if not dqkv.is_contiguous():
        raise ValueError("dqkv must be contiguous")
    if dqkv.numel() != sizes[0] * w.shape[0]:
        raise ValueError("dqkv must hold 3*NH*HD values per token of x")
    outputs = [("dlora_a", dlora_a, bf16, lora_a.shape), ("dlora_b", dlora_b, bf16, lora_b.shape)]
    if dx is not None:
        outputs.append(("dx", dx, bf16, x.shape))
    _check_on_device(outputs)
    work = _workspace(work, max(0, lib.na3d_lora_workspace(*sizes, 1)), x, stream)
    rc = lib.na3d_lora_qkv_proj_bwd(dqkv.data_ptr(), x.data_ptr(), w.data_ptr(), lora_a.data_ptr(),
                                    lora_b.data_ptr(), scaling.data_ptr(), offsets.data_ptr(), adapter.data_ptr(),
                                    None if dx is None else dx.data_ptr(), dlora_a.data_ptr(), dlora_b.data_ptr(),
                                    work.data_ptr(), *sizes, _stream_handle(stream))
    if rc != NA3D_OK:
        raise NA3DError(rc, "na3d_lora_qkv_proj_bwd")


def na3d_rope_table(grid, rope_dims, theta=10000.0, offset=(0.0, 0.0, 0.0), scale=(1.0, 1.0, 1.0), device=None,
                    stream=None):
    """The fp32 table of cosines and sines for ``na3d_norm_rope`` on a grid
    (T, H, W), ``rope_dims`` = (RT, RH, RW) values of a head turning with each
    axis: (T*RT + H*RH + W*RW) / 2 rows of (cos, sin) of the angles
    (offset + scale * position) * theta**(-2 i / R), axis after axis, position
    after position. Made once for a grid and kept; a table of other frequencies
    is filled in the same layout. On the current CUDA device."""
    lib = _lib if _lib is not None else load_library()
    torch = _torch_module()
    T, H, W = (int(x) for x in grid)
    RT, RH, RW = (int(x) for x in rope_dims)
    if min(T, H, W) < 1 or min(RT, RH, RW) < 0 or (RT | RH | RW) & 1 or not RT + RH + RW:
        raise NA3DError(2, "na3d_rope_table")
    table = _empty_on(stream, device if device is not None else torch.device("cuda", torch.cuda.current_device()),
                      ((T * RT + H * RH + W * RW) // 2, 2), torch.float32)
    if table.get_device() != torch.cuda.current_device():
        raise TypeError("device must be the current CUDA device")
    rc = lib.na3d_rope_table(table.data_ptr(), T, H, W, RT, RH, RW, theta, *offset, *scale, _stream_handle(stream))
    if rc != NA3D_OK:
        raise NA3DError(rc, "na3d_rope_table")
    return table


def _rope_call(q, k, q_rows, k_rows, q_weight, k_weight, table, rope_dims):
    """What both directions of the norm and rotation check: (sizes, strides, weight and
    table pointers). q_rows, k_rows: the (name, tensor) of q's and k's shape besides q and k."""
    torch = _torch_module()
    dev = _device()
    Tensor, bf16 = torch.Tensor, torch.bfloat16
    if not isinstance(q, Tensor):
        raise TypeError("q must be a torch.Tensor")
    shape = q.shape
    if len(shape) != 6:
        raise ValueError("q must have a 6-D (B,T,H,W,NH,HD) shape")
    B, T, H, W, NH, HD = shape
    if k is None:
        if k_weight is not None or any(t is not None for _, t in k_rows):
            raise ValueError("k's tensors need k")
        k_shape, NKV = None, 0
        sides = ((shape, (("q", q), *q_rows)),)
    else:
        if not isinstance(k, Tensor):
            raise TypeError("k must be a torch.Tensor")
        k_shape = k.shape
        if len(k_shape) != 6 or k_shape[:4] != shape[:4] or k_shape[5] != HD:
            raise ValueError("k must have a 6-D (B,T,H,W,NKV,HD) shape that goes with q's")
        NKV = k_shape[4]
        sides = ((shape, (("q", q), *q_rows)), (k_shape, (("k", k), *k_rows)))
    strides = []
    for want, tensors in sides:
        was = row = None
        for name, t in tensors:
            if not isinstance(t, Tensor):
                raise TypeError(f"{name} must be a torch.Tensor")
            if t.dtype is not bf16 or t.get_device() != dev:
                raise TypeError(f"{name} must be a bfloat16 tensor on the current CUDA device")
            if t.shape != want:
                raise ValueError(f"{name} must have the shape {tuple(want)}, not {tuple(t.shape)}")
            st = t.stride()
            if st != was:
                was, row = st, _token_stride(name, t)
            strides.append(row)
    if k is None:
        strides += [0] * len(strides)
    n = len(strides) // 2
    RT, RH, RW = rope_dims
    pointers = [None, None, None]
    if q_weight is not None:
        _check_one(torch, dev, "q_weight", q_weight, bf16, (HD,))
        pointers[0] = q_weight.data_ptr()
    if k_weight is not None:
        _check_one(torch, dev, "k_weight", k_weight, bf16, (HD,))
        pointers[1] = k_weight.data_ptr()
    if table is not None:
        _check_one(torch, dev, "table", table, torch.float32, ((T * RT + H * RH + W * RW) // 2, 2))
        pointers[2] = table.data_ptr()
    sizes = (B, T, H, W, NH, NKV, HD, int(RT), int(RH), int(RW))
    return sizes, [x for i in range(n) for x in (strides[i], strides[n + i])], pointers


def _at(t):
    return None if t is None else t.data_ptr()


def na3d_norm_rope(q, k, q_out, k_out, q_weight=None, k_weight=None, table=None, rope_dims=(0, 0, 0), norm=True,
                   q_eps=1e-6, k_eps=1e-6, q_scale=1.0, interleaved=True, stream=None) -> None:
    """q_out, k_out = the heads of q and k, RMS-normed (``norm``; ``q_weight``,
    ``k_weight``: bf16 (HD,) or None for ones) and turned by their position on the
    grid (see ``na3d_norm_rope`` in include/na3d.h). q and q_out: (B, T, H, W, NH,
    HD), k and k_out: (B, T, H, W, NKV, HD) or both None; all may be views with a
    token stride, an output may be its own input. ``table``: what
    ``na3d_rope_table`` made for (T, H, W) and ``rope_dims`` = (RT, RH, RW), the
    values of a head that turn with each axis, or None with (0, 0, 0). Pairs are
    neighbours (``interleaved``) or the halves of the values that turn. ``q_scale``
    multiplies q_out: HD**-0.5 makes it what the attention wants. For a q that
    ``na3d_qkv_proj`` scaled by HD**-0.5, q_eps = eps / HD gives the norm of the
    unscaled q. Autograd does not see the call: the gradients come from
    ``na3d_norm_rope_bwd``."""
    lib = _lib if _lib is not None else load_library()
    sizes, strides, at = _rope_call(q, k, (("q_out", q_out),), (("k_out", k_out),), q_weight, k_weight, table, rope_dims)
    rc = lib.na3d_norm_rope(q.data_ptr(), _at(k), q_out.data_ptr(), _at(k_out), *at, *sizes, *strides,
                            1 if norm else 0, q_eps, k_eps, q_scale, 1 if interleaved else 0, _stream_handle(stream))
    if rc != NA3D_OK:
        raise NA3DError(rc, "na3d_norm_rope")


@functools.lru_cache(maxsize=64)
def _rope_need(head_dim) -> int:
    return load_library().na3d_norm_rope_workspace(head_dim)


def na3d_norm_rope_workspace(head_dim) -> int:
    """Bytes of workspace that ``na3d_norm_rope_bwd`` uses for the weights' gradients."""
    need = _rope_need(int(head_dim))
    if need < 0:
        raise ValueError("head_dim must be a power of two from 16 to 512")
    return need


def na3d_norm_rope_bwd(q, k, dq_out, dk_out, dq, dk, dq_weight=None, dk_weight=None, q_weight=None, k_weight=None,
                       table=None, rope_dims=(0, 0, 0), norm=True, q_eps=1e-6, k_eps=1e-6, q_scale=1.0,
                       interleaved=True, work=None, stream=None) -> None:
    """dq, dk = the gradients of ``na3d_norm_rope`` with respect to q and k, for
    those of its outputs (``dq_out``, ``dk_out``); ``dq_weight``, ``dk_weight``: fp32
    (HD,) for the weights' gradients, or None. dq may be dq_out or q, dk dk_out or
    k; all may be views with a token stride. q and k are the forward pass's inputs,
    the other arguments the forward pass's. ``work``: a tensor of
    ``na3d_norm_rope_workspace`` bytes, kept by the caller (one call at a time);
    None takes one that the binding keeps (for this thread and the current stream;
    a call with a ``stream`` or under capture allocates its own)."""
    lib = _lib if _lib is not None else load_library()
    sizes, strides, at = _rope_call(q, k, (("dq_out", dq_out), ("dq", dq)), (("dk_out", dk_out), ("dk", dk)), q_weight,
                                    k_weight, table, rope_dims)
    if dq_weight is not None or dk_weight is not None:
        for name, w in (("dq_weight", dq_weight), ("dk_weight", dk_weight)):
            if w is not None:
                _check_one(_torch, _device(), name, w, _torch.float32, (sizes[6],))
        work = _workspace(work, max(0, _rope_need(sizes[6])), q, stream)
    rc = lib.na3d_norm_rope_bwd(q.data_ptr(), _at(k), dq_out.data_ptr(), _at(dk_out), dq.data_ptr(), _at(dk),
                                _at(dq_weight), _at(dk_weight), *at, _at(work), *sizes, *strides, 1 if norm else 0, q_eps,
                                k_eps, q_scale, 1 if interleaved else 0, _stream_handle(stream))
    if rc != NA3D_OK:
        raise NA3DError(rc, "na3d_norm_rope_bwd")


def _state_stride(name, t) -> int:
    """Elements between consecutive states of a (B,S,NKV,HD) view whose heads are packed."""
    st, sh = t.stride(), t.shape
    if st[3] != 1 or (sh[2] > 1 and st[2] != sh[3]):
        raise ValueError(f"{name}: heads must be packed (strides [..., HD, 1])")
    if sh[1] > 1:
        if sh[0] > 1 and st[0] != sh[1] * st[1]:
            raise ValueError(f"{name}: states must share one token stride")
        return st[1]
    return st[0] if sh[0] > 1 else sh[2] * sh[3]


def _cross_call(q, rows, states, doc, kv_doc):
    """What both directions of the attention to other states check: (sizes, token
    strides of q, rows and states in turn, pointers of doc and kv_doc). rows: (name,
    tensor) like q; states: (name, tensor) of k's shape, k first."""
    torch = _torch_module()
    dev = _device()
    Tensor, bf16 = torch.Tensor, torch.bfloat16
    k = states[0][1]
    if not isinstance(q, Tensor) or not isinstance(k, Tensor):
        raise TypeError("q and k must be a torch.Tensor")
    shape, k_shape = q.shape, k.shape
    if len(shape) != 6 or len(k_shape) != 4:
        raise ValueError("q must be 6-D (B,T,H,W,NH,HD), k and v 4-D (B,S,NKV,HD)")
    B, T, H, W, NH, HD = shape
    strides, row, want, was = [], _token_stride, shape, None
    for name, t in (("q", q), *rows, *states):
        if t is k:
            row, want, was = _state_stride, k_shape, None
        if not isinstance(t, Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dtype is not bf16 or t.get_device() != dev:
            raise TypeError(f"{name} must be a bfloat16 tensor on the current CUDA device")
        if t.shape != want:
            raise ValueError(f"{name} must have the shape of {'q' if want is shape else 'k'}")
        st = t.stride()
        if st != was:
            was, step = st, row(name, t)
        strides.append(step)
    if k_shape[0] != B or k_shape[3] != HD:
        raise ValueError("q and k must agree on B and HD")
    at = [None, None]
    if doc is not None:
        _check_one(torch, dev, "doc", doc, torch.int32, (B, T, H, W))
        at[0] = doc.data_ptr()
    if kv_doc is not None:
        _check_one(torch, dev, "kv_doc", kv_doc, torch.int32, (B, k_shape[1]))
        at[1] = kv_doc.data_ptr()
    return (B, T * H * W, k_shape[1], NH, k_shape[2], HD), strides, at


@functools.lru_cache(maxsize=256)
def _cross_need(B, L, S, num_heads, kv_heads, head_dim, backward) -> int:
    """What the library answers of these sizes (asking takes a microsecond of a call's twenty)."""
    return load_library().na3d_cross_workspace(B, L, S, num_heads, kv_heads, head_dim, backward)


def na3d_cross_workspace(B, L, S, num_heads, kv_heads, head_dim, backward=False) -> int:
    """Bytes of workspace of ``na3d_cross_fwd``, or of ``na3d_cross_bwd``, for L = T*H*W tokens an entry."""
    need = int(load_library().na3d_cross_workspace(B, L, S, num_heads, kv_heads, head_dim, 1 if backward else 0))
    if need < 0:
        raise ValueError("sizes that na3d_cross_fwd does not take")
    return need


def _call_cross_fwd(q, k, v, out, lse, sizes, strides, pointers, work, stream) -> None:
    """The call behind na3d_cross_fwd: all but work is checked."""
    lib = _lib if _lib is not None else load_library()
    need = _cross_need(*sizes, 0)
    if need > 0:
        work = _workspace(work, need, q, stream)
    rc = lib.na3d_cross_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), _at(lse), _at(work), *sizes,
                            *strides, *pointers, _stream_handle(stream))
    if rc != NA3D_OK:
        raise NA3DError(rc, "na3d_cross_fwd")


def na3d_cross_fwd(q, k, v, out, lse=None, doc=None, kv_doc=None, work=None, stream=None) -> None:
    """Attention of a grid's tokens q (B, T, H, W, NH, HD) to states k, v (B, S,
    NKV, HD) of another length, e.g. a prompt's (see ``na3d_cross_fwd`` in
    include/na3d.h). q is scaled by HD**-0.5; NKV divides NH, heads of q share those
    of k and v in runs of NH / NKV; q, k and v may be views with a token stride, e.g.
    ``kv[:, :, 0]`` of a fused (B, S, 2, NKV, HD) projection. ``doc``: int32 (B, T, H,
    W), ``kv_doc``: int32 (B, S); a token sees the states of its document, None is
    document 0 for all, negative ones are padding. ``out`` is contiguous; ``lse``,
    where given, receives the fp32 (B, T, H, W, NH) log-sum-exp. HD up to 128.
    ``work``: a tensor of ``na3d_cross_workspace`` bytes, kept by the caller (one
    call at a time); None takes one that the binding keeps where one is needed (for
    this thread and the current stream; a call with a ``stream`` or under capture
    allocates its own). Autograd does not see the call: the gradients come from
    ``na3d_cross_bwd``."""
    sizes, (q_ts, _, *kv_ts), pointers = _cross_call(q, (("out", out),), (("k", k), ("v", v)), doc, kv_doc)
    if not out.is_contiguous():
        raise ValueError("out must be contiguous")
    if lse is not None:
        _check_one(_torch, _device(), "lse", lse, _torch.float32, q.shape[:5])
    _call_cross_fwd(q, k, v, out, lse, sizes, (q_ts, *kv_ts), pointers, work, stream)


def na3d_cross_attention(q, k, v, doc=None, kv_doc=None, return_lse=False, stream=None):
    """``na3d_cross_fwd`` into a new tensor: returns out, or (out, lse) where
    ``return_lse`` is true (what ``na3d_cross_bwd`` needs)."""
    torch = _torch_module()
    sizes, strides, pointers = _cross_call(q, (), (("k", k), ("v", v)), doc, kv_doc)
    shape, device = q.shape, q.device
    out = _empty_on(stream, device, shape, torch.bfloat16)
    lse = _empty_on(stream, device, shape[:5], torch.float32) if return_lse else None
    _call_cross_fwd(q, k, v, out, lse, sizes, strides, pointers, None, stream)
    return (out, lse) if return_lse else out


def na3d_cross_bwd(q, k, v, out, lse, dout, dq, dk, dv, doc=None, kv_doc=None, work=None, stream=None) -> None:
    """dq, dk, dv = the gradients of ``na3d_cross_fwd`` for the gradient ``dout`` of
    its output. ``out`` and ``lse`` are what the forward pass wrote; the other
    arguments are the forward pass's. dq, dk and dv may be views with a token stride,
    e.g. the blocks of a fused gradient. ``work``: a tensor of
    ``na3d_cross_workspace`` bytes with ``backward=True``, as there."""
    lib = _lib if _lib is not None else load_library()
    sizes, (q_ts, _, _, dq_ts, k_ts, v_ts, dk_ts, dv_ts), pointers = _cross_call(
        q, (("out", out), ("dout", dout), ("dq", dq)), (("k", k), ("v", v), ("dk", dk), ("dv", dv)), doc, kv_doc)
    if not (out.is_contiguous() and dout.is_contiguous()):
        raise ValueError("out and dout must be contiguous")
    _check_one(_torch, _device(), "lse", lse, _torch.float32, q.shape[:5])
    work = _workspace(work, max(0, _cross_need(*sizes, 1)), q, stream)
    rc = lib.na3d_cross_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), dout.data_ptr(),
                            dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), work.data_ptr(), *sizes,
                            q_ts, k_ts, v_ts, dq_ts, dk_ts, dv_ts, *pointers, _stream_handle(stream))
    if rc != NA3D_OK:
        raise NA3DError(rc, "na3d_cross_bwd")


def na3d_plan(T, H, W, NH, HD, KT, KH, KW) -> dict:
    """The tiling ``na3d_fwd`` uses for this problem (host only, no GPU)."""
    info = PlanInfo()
    rc = load_library().na3d_plan(T, H, W, NH, HD, KT, KH, KW, ctypes.byref(info))
    if rc != NA3D_OK:
        raise NA3DError(rc, "na3d_plan")
    return {name: getattr(info, name) for name, _ in PlanInfo._fields_}


def na3d_device_status(stream=None) -> int:
    """Synchronize ``stream``; NA3D_ERR_DEVICE_TIMEOUT if a kernel wait gave up."""
    return int(load_library().na3d_device_status(_stream_handle(stream)))
