"""The packed-batch entry points refuse bad arguments before anything is
enqueued (C statuses and the binding's exceptions); no GPU needed."""
import ctypes

import pytest
import torch

import neighborhood_attention_video_gb300 as na
from neighborhood_attention_video_gb300 import build as na_build

OK, ERR_NULL, ERR_SHAPE, ERR_KERNEL, ERR_HEAD_DIM, ERR_ALIGN, ERR_ALIAS = 0, 1, 2, 3, 4, 5, 6
ERR_OVERFLOW, ERR_CUDA, ERR_UNSUPPORTED = 7, 9, 11
P = ctypes.c_void_p
BASE, STEP = 1 << 30, 1 << 26      # invalid calls only: these addresses are never touched


@pytest.fixture(scope="module")
def lib():
    na_build.build()
    return na.load_library()


def fwd(lib, dims=(1, 4, 8, 16, 2, 32), kernel=(3, 5, 5), strides=None, softcap=0.0, **ptrs):
    names = ("q", "k", "v", "out", "lse")
    at = {n: BASE + i * STEP for i, n in enumerate(names)}
    at.update(slopes=None, doc=None, prefix=None)
    at.update(ptrs)
    nhd = dims[4] * dims[5]
    return lib.na3d_scored_fwd(*[P(at[n]) for n in names], *dims, *kernel, *(strides or (nhd,) * 3), softcap,
                               P(at["slopes"]), P(at["doc"]), P(at["prefix"]), None)


@pytest.mark.parametrize("code,change", [
    (ERR_SHAPE, dict(dims=(0, 4, 8, 16, 2, 32))),
    (ERR_KERNEL, dict(kernel=(3, 4, 5))),
    (ERR_KERNEL, dict(kernel=(5, 5, 5))),
    (ERR_HEAD_DIM, dict(dims=(1, 4, 8, 16, 2, 48))),
    (ERR_UNSUPPORTED, dict(dims=(1, 4, 8, 16, 2, 256))),
    (ERR_UNSUPPORTED, dict(softcap=-1.0)),
    (ERR_UNSUPPORTED, dict(softcap=float("nan"))),
    (ERR_UNSUPPORTED, dict(softcap=float("inf"))),
    (ERR_UNSUPPORTED, dict(softcap=1e-4)),
    (ERR_OVERFLOW, dict(dims=(1 << 40, 4, 8, 16, 2, 32))),
    (ERR_NULL, dict(q=0)),
    (ERR_NULL, dict(out=0)),
    (ERR_ALIGN, dict(k=BASE + STEP + 8)),
    (ERR_ALIGN, dict(lse=BASE + 4 * STEP + 2)),
    (ERR_ALIGN, dict(doc=BASE + 5 * STEP + 1)),
    (ERR_SHAPE, dict(strides=(56, 64, 64))),
    (ERR_ALIGN, dict(strides=(64, 68, 64))),
    (ERR_ALIAS, dict(out=BASE + STEP + 16)),
    (ERR_ALIAS, dict(lse=BASE + 3 * STEP + 64)),
    (ERR_ALIAS, dict(doc=BASE + 3 * STEP + 64)),
])
def test_scored_fwd_refusals(lib, code, change):
    assert fwd(lib, **change) == code


def bwd(lib, dims=(1, 4, 8, 16, 2, 32), strides=None, **ptrs):
    names = ("q", "k", "v", "out", "lse", "dout", "dq", "dk", "dv", "work")
    at = {n: BASE + i * STEP for i, n in enumerate(names)}
    at.update(ptrs)
    return lib.na3d_scored_bwd(*[P(at[n]) for n in names], *dims, 3, 5, 5, *(strides or (dims[4] * dims[5],) * 6), 0.0,
                               None, None, None, None)


@pytest.mark.parametrize("code,change", [
    (ERR_NULL, dict(lse=0)),
    (ERR_NULL, dict(work=0)),
    (ERR_ALIGN, dict(dq=BASE + 6 * STEP + 8)),
    (ERR_ALIAS, dict(dq=BASE)),                                       # over q
    (ERR_ALIAS, dict(dk=BASE + 6 * STEP + 128)),                      # inside dq
    (ERR_ALIAS, dict(work=BASE + 8 * STEP)),                          # over dv
    # the blocks of one fused gradient, the second shifted into the first
    (ERR_ALIAS, dict(strides=(64,) * 3 + (192,) * 3, dk=BASE + 6 * STEP + 112, dv=BASE + 6 * STEP + 256)),
    # ... or their rows wrapping into the next token's
    (ERR_ALIAS, dict(strides=(64,) * 3 + (144,) * 3, dk=BASE + 6 * STEP + 176, dv=BASE + 8 * STEP)),
])
def test_scored_bwd_refusals(lib, code, change):
    assert bwd(lib, **change) == code


def test_scored_bwd_takes_a_fused_gradient(lib):
    """The three blocks of a (..., 3, NH, HD) gradient pass every check; the call
    then fails for want of a GPU."""
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    at = BASE + 6 * STEP
    assert bwd(lib, strides=(64,) * 3 + (192,) * 3, dk=at + 128, dv=at + 256) == ERR_CUDA
    assert fwd(lib) == ERR_CUDA and fwd(lib, lse=0) == ERR_CUDA and fwd(lib, softcap=30.0) == ERR_CUDA


def test_windows_without_a_plan_are_refused(lib):
    """... as unsupported, before anything is enqueued, not as a CUDA error."""
    wide, kernel = (1, 1, 600, 600, 1, 64), (1, 511, 511)
    far = {n: (i + 1) << 36 for i, n in enumerate(("q", "k", "v", "out", "lse", "dout", "dq", "dk", "dv", "work"))}
    assert fwd(lib, wide, kernel, **{n: far[n] for n in ("q", "k", "v", "out", "lse")}) == ERR_UNSUPPORTED
    call = lib.na3d_scored_bwd
    assert call(*[P(x) for x in far.values()], *wide, *kernel, *(64,) * 6, 0.0, None, None, None, None) == ERR_UNSUPPORTED
    many = (1 << 30, 1, 1, 1, 4, 16)
    assert fwd(lib, many, (1, 1, 1), **{n: (i + 1) << 40 for i, n in enumerate(("q", "k", "v", "out", "lse"))}) == ERR_UNSUPPORTED


def lora(lib, backward, sizes=(100, 64, 2, 32, 16, 3, 2), **ptrs):
    names = ("x", "w", "bias", "a", "b", "scaling", "offsets", "adapter", "qkv", "work")
    if backward:
        names = ("dqkv", "x", "w", "a", "b", "scaling", "offsets", "adapter", "dx", "da", "db", "work")
    at = {n: BASE + i * STEP for i, n in enumerate(names)}
    at.update(ptrs)
    call = lib.na3d_lora_qkv_proj_bwd if backward else lib.na3d_lora_qkv_proj
    return call(*[P(at[n]) for n in names], *sizes, None)


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("code,change", [
    (ERR_SHAPE, dict(sizes=(0, 64, 2, 32, 16, 3, 2))),
    (ERR_SHAPE, dict(sizes=(100, 64, 2, 32, 0, 3, 2))),
    (ERR_SHAPE, dict(sizes=(100, 64, 2, 32, 16, 0, 2))),
    (ERR_SHAPE, dict(sizes=(100, 64, 2, 32, 16, 3, 0))),
    (ERR_HEAD_DIM, dict(sizes=(100, 64, 2, 48, 16, 3, 2))),
    (ERR_ALIGN, dict(sizes=(100, 60, 2, 32, 16, 3, 2))),
    (ERR_ALIGN, dict(sizes=(100, 64, 2, 32, 12, 3, 2))),
    (ERR_UNSUPPORTED, dict(sizes=(100, 64, 2, 32, 136, 3, 2))),
    (ERR_UNSUPPORTED, dict(sizes=(100, 64, 2, 32, 16, 101 + (1 << 20), 2))),
    (ERR_OVERFLOW, dict(sizes=(1 << 31, 64, 2, 32, 16, 3, 2))),
    (ERR_OVERFLOW, dict(sizes=(100, 64, 1 << 27, 32, 16, 3, 2))),
    (ERR_NULL, dict(x=0)),
    (ERR_NULL, dict(adapter=0)),
    (ERR_NULL, dict(work=0)),
    (ERR_ALIGN, dict(a=BASE + 20 * STEP + 8)),
    (ERR_ALIGN, dict(work=BASE + 20 * STEP + 8)),
    (ERR_ALIGN, dict(offsets=BASE + 20 * STEP + 2)),
])
def test_lora_refusals(lib, backward, code, change):
    assert lora(lib, backward, **change) == code


def test_lora_alias_refusals(lib):
    assert lora(lib, False, qkv=BASE + 16) == ERR_ALIAS                     # over x
    assert lora(lib, False, work=BASE + 8 * STEP) == ERR_ALIAS              # over qkv
    assert lora(lib, True, dx=BASE + STEP) == ERR_ALIAS                     # over x
    assert lora(lib, True, da=BASE + 10 * STEP) == ERR_ALIAS                # over db
    if not torch.cuda.is_available():
        assert lora(lib, False) == ERR_CUDA and lora(lib, True, dx=0) == ERR_CUDA
        assert lora(lib, False, bias=0) == ERR_CUDA


def test_workspace_sizes(lib):
    assert na.na3d_scored_bwd_workspace(2, 3, 4, 5, 6) >= 4 * 720
    assert na.na3d_lora_workspace(100, 64, 2, 32, 16, 3, 2) > 0
    with pytest.raises(ValueError):
        na.na3d_scored_bwd_workspace(2, 0, 4, 5, 6)
    with pytest.raises(ValueError):
        na.na3d_lora_workspace(100, 64, 2, 32, 12, 3, 2)


def test_lora_workspace_past_int64_is_refused(lib):
    """The adapters' sums of these sizes hold 2^60 values, each size by itself in range."""
    sizes = (100, (1 << 31) - 8, 1, 16, 128, 3, 1 << 23)
    assert lora(lib, True, sizes=sizes) == ERR_OVERFLOW
    with pytest.raises(ValueError):
        na.na3d_lora_workspace(*sizes, backward=True)


def test_binding_wants_device_tensors():
    x = torch.zeros(1, 4, 8, 16, 2, 32, dtype=torch.bfloat16)
    lse = torch.zeros(1, 4, 8, 16, 2)
    with pytest.raises(TypeError):
        na.na3d_scored_fwd(x, x, x, x.clone(), (3, 5, 5))
    with pytest.raises(TypeError):
        na.na3d_scored_attention(x, x, x, (3, 5, 5))
    with pytest.raises(TypeError):
        na.na3d_scored_bwd(x, x, x, x, lse, x, x, x, x, (3, 5, 5))
    ids = torch.zeros(2, dtype=torch.int32)
    y = torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        na.na3d_lora_qkv_proj(y, y, None, y[None], y[None], lse, ids, ids[:1], y, 1, 16)
    with pytest.raises(ValueError):
        na.na3d_lora_qkv_proj(y, y, None, y, y[None], lse, ids, ids[:1], y, 1, 16)


def test_qkv_views_of_any_array():
    """Views of whatever indexes like a tensor, arrays of the oracle's inputs among them."""
    x = torch.arange(2 * 3 * 2 * 4).reshape(2, 3, 2, 4)
    for a in (x, x.numpy()):
        views = na.qkv_views(a)
        for i, v in enumerate(views):
            assert type(v) is type(a) and tuple(v.shape) == (2, 2, 4) and (v == a[:, i]).all()
            v[0, 0, 0] = -1
            assert a[0, i, 0, 0] == -1


@pytest.mark.parametrize("cut", [(0, 3, 1, 1), (0, 3, 2, 1), (0, 1, 1, 4), (0, 3, 1, 4), (0, 1, 5, 1), (2, 1, 1, 1), (0, 1, 1, 1),
                                 (2, 3, 5, 7), (0, 3, 5, 7)])
@pytest.mark.parametrize("H0", [5, 1])
def test_token_stride_of_cut_grids(cut, H0):
    """The token stride of a view is that of its axes of more than one position: an axis
    of one says nothing. Where positions share no stride the view is refused."""
    B, T, H, W = (n or 1 for n in cut)
    H = min(H, H0)
    x = torch.zeros(2, 3, H0, 7, 2, 16)[:B, :T, :H, :W]
    offsets = [sum(i * s for i, s in zip(at, x.stride())) for at in
               ((b, t, h, w) for b in range(B) for t in range(T) for h in range(H) for w in range(W))]
    steps = {b - a for a, b in zip(offsets, offsets[1:])}
    if len(steps) > 1:
        with pytest.raises(ValueError):
            na._token_stride("x", x)
    else:
        assert na._token_stride("x", x) == (steps.pop() if steps else 2 * 16)


def test_token_stride_of_repeated_positions():
    """Positions that share memory have no stride that the library takes: 0, or none at all."""
    x = torch.zeros(1, 1, 1, 1, 2, 16)
    for shape in ((1, 1, 1, 4, 2, 16), (1, 1, 3, 4, 2, 16), (2, 1, 1, 1, 2, 16)):
        assert na._token_stride("x", x.expand(shape)) == 0
    with pytest.raises(ValueError):
        na._token_stride("x", torch.zeros(1, 1, 3, 1, 2, 16).expand(1, 1, 3, 4, 2, 16))
