"""Python binding of the GB300 NA3D forward library (``libna3d.so``).

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI declared in ``include/na3d.h``. There is no CPU or
PyTorch fallback; if the library has not been built, importing works but any
call raises ``NA3DUnavailable``.

PyTorch is used for device memory and streams only.
"""
from __future__ import annotations

import ctypes
import os
import threading

__all__ = [
    "NA3DError", "NA3DUnavailable", "na3d_attention", "na3d_fwd", "na3d_fwd_strided", "na3d_fwd_region",
    "na3d_qkv_proj", "qkv_views", "na3d_scored_fwd", "na3d_scored_attention", "na3d_scored_bwd",
    "na3d_lora_qkv_proj", "na3d_lora_qkv_proj_bwd", "na3d_lora_workspace",
    "na3d_scored_bwd_workspace", "na3d_status_string", "na3d_plan",
    "na3d_device_status", "library_path", "load_library", "EXPORTED_SYMBOLS",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libna3d.so")
EXPORTED_SYMBOLS = ("na3d_fwd", "na3d_fwd_strided", "na3d_fwd_region", "na3d_qkv_proj",
                    "na3d_scored_fwd", "na3d_scored_bwd", "na3d_scored_bwd_workspace",
                    "na3d_lora_qkv_proj", "na3d_lora_qkv_proj_bwd", "na3d_lora_workspace",
                    "na3d_selftest_withhold", "na3d_status_string", "na3d_plan",
                    "na3d_device_status")

NA3D_OK = 0
_I64 = ctypes.c_int64
_P = ctypes.c_void_p
_F32 = ctypes.c_float
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
    lib.na3d_selftest_withhold.argtypes = [_P, _P, _P, _P] + [_I64] * 10 + [_P]
    lib.na3d_selftest_withhold.restype = ctypes.c_int
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


def _torch_module():
    global _torch, _cuda_ok
    if _torch is None:
        import torch
        _torch = torch
        _cuda_ok = torch.cuda.is_available()
    return _torch


def _check_bf16_on_device(tensors):
    """Each (name, tensor) is a bf16 tensor on the current CUDA device: the
    kernels get raw pointers, so a host or other-device tensor must not pass."""
    torch = _torch_module()
    dev = torch.cuda.current_device() if _cuda_ok else -2
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
            return raw(torch.cuda.current_device())
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
    dev = torch.cuda.current_device() if _cuda_ok else -2
    for name, t, dtype, shape in tensors:
        _check_one(torch, dev, name, t, dtype, shape)


def _check_bf16_of_shape(shape, names, tensors):
    """The tensors are bf16, of one 6-D shape, on the current CUDA device."""
    torch = _torch_module()
    dev, bf16 = torch.cuda.current_device() if _cuda_ok else -2, torch.bfloat16
    for name, t in zip(names, tensors):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dtype is not bf16 or t.get_device() != dev:
            raise TypeError(f"{name} must be a bfloat16 tensor on the current CUDA device")
        if t.shape != shape:
            raise ValueError(f"{name} must have the (B,T,H,W,NH,HD) shape of q")
    if len(shape) != 6:
        raise ValueError("q must have a 6-D (B,T,H,W,NH,HD) shape")


def _empty(stream, like, shape, dtype):
    """A new tensor on the device of `like`, allocated on the stream that the
    call uses, so that the allocator may reuse its memory only behind the call."""
    torch = _torch_module()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


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
    dev = torch.cuda.current_device() if _cuda_ok else -2
    if not isinstance(work, torch.Tensor) or work.get_device() != dev or not work.is_contiguous():
        raise TypeError("work must be a contiguous tensor on the current CUDA device")
    if work.numel() * work.element_size() < need:
        raise ValueError(f"work must hold {need} bytes")
    return work


def _scored_options(shape, softcap, slopes, doc, prefix):
    """The score arguments of the na3d_scored_ calls, checked: (softcap, the
    three pointers or None)."""
    torch = _torch_module()
    dev = torch.cuda.current_device() if _cuda_ok else -2
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
