"""The entry points of the norm, rotation and cross attention refuse bad arguments
before anything is enqueued (C statuses and the binding's exceptions); no GPU needed."""
import ctypes

import pytest
import torch

import neighborhood_attention_video_gb300 as na
from neighborhood_attention_video_gb300 import build as na_build

OK, ERR_NULL, ERR_SHAPE, ERR_HEAD_DIM, ERR_ALIGN, ERR_ALIAS = 0, 1, 2, 4, 5, 6
ERR_OVERFLOW, ERR_CUDA, ERR_UNSUPPORTED = 7, 9, 11
P = ctypes.c_void_p
BASE, STEP = 1 << 30, 1 << 26      # invalid calls only: these addresses are never touched
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    na_build.build()
    return na.load_library()


def rope(lib, backward, dims=(1, 4, 8, 16, 2, 2, 32), turned=(8, 12, 12), strides=None, norm=1, q_eps=1e-6, k_eps=1e-6,
         q_scale=1.0, interleaved=1, **ptrs):
    names = ("q", "k", "q_out", "k_out", "q_weight", "k_weight", "table")
    if backward:
        names = ("q", "k", "dq_out", "dk_out", "dq", "dk", "dqw", "dkw", "q_weight", "k_weight", "table", "work")
    at = {n: BASE + i * STEP for i, n in enumerate(names)}
    at.update(ptrs)
    rows = (dims[4] * dims[6], dims[5] * dims[6])
    call = lib.na3d_norm_rope_bwd if backward else lib.na3d_norm_rope
    return call(*[P(at[n]) for n in names], *dims, *turned, *(strides or rows * (3 if backward else 2)), norm, q_eps, k_eps,
                q_scale, interleaved, None)


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("code,change", [
    (ERR_SHAPE, dict(dims=(0, 4, 8, 16, 2, 2, 32))),
    (ERR_SHAPE, dict(dims=(1, 4, 8, 16, 0, 2, 32))),
    (ERR_SHAPE, dict(dims=(1, 4, 8, 16, 2, -1, 32))),
    (ERR_SHAPE, dict(turned=(8, 12, 14))),
    (ERR_SHAPE, dict(turned=(8, 11, 12))),
    (ERR_SHAPE, dict(turned=(-2, 12, 12))),
    (ERR_HEAD_DIM, dict(dims=(1, 4, 8, 16, 2, 2, 48))),
    (ERR_HEAD_DIM, dict(dims=(1, 4, 8, 16, 2, 2, 8))),
    (ERR_UNSUPPORTED, dict(dims=(1, 4, 8, 16, 2, 2, 1024))),
    (ERR_UNSUPPORTED, dict(interleaved=0, turned=(8, 12, 10))),
    (ERR_UNSUPPORTED, dict(q_eps=0.0)),
    (ERR_UNSUPPORTED, dict(k_eps=-1.0)),
    (ERR_UNSUPPORTED, dict(q_eps=NAN)),
    (ERR_UNSUPPORTED, dict(k_eps=INF)),
    (ERR_UNSUPPORTED, dict(q_scale=INF)),
    (ERR_UNSUPPORTED, dict(norm=0)),                                          # with weights
    (ERR_OVERFLOW, dict(dims=(1 << 20, 1 << 5, 8, 16, 2, 2, 32))),
    (ERR_OVERFLOW, dict(dims=(1 << 62, 4, 8, 16, 2, 2, 32))),
    (ERR_OVERFLOW, dict(dims=(1, 4, 8, 16, 1 << 27, 2, 32))),
    (ERR_OVERFLOW, dict(dims=(1, 1 << 27, 1, 1, 1, 1, 32))),                  # the table
    (ERR_NULL, dict(q=0)),
    (ERR_NULL, dict(k=0)),
    (ERR_NULL, dict(table=0)),
    (ERR_ALIGN, dict(q=BASE + 8)),
    (ERR_ALIGN, dict(q_weight=BASE + 20 * STEP + 8)),
    (ERR_ALIGN, dict(table=BASE + 20 * STEP + 4)),
])
def test_norm_rope_refusals(lib, backward, code, change):
    assert rope(lib, backward, **change) == code


@pytest.mark.parametrize("code,change", [
    (ERR_NULL, dict(q_out=0)),
    (ERR_NULL, dict(k_out=0)),
    (ERR_SHAPE, dict(strides=(56, 64, 64, 64))),
    (ERR_ALIGN, dict(strides=(64, 68, 64, 64))),
    (ERR_ALIAS, dict(q_out=BASE + 16)),                                       # beside q
    (ERR_ALIAS, dict(q_out=BASE, strides=(64, 64, 128, 64))),                 # in place with another stride
    (ERR_ALIAS, dict(q_out=BASE + STEP)),                                     # over k
    (ERR_ALIAS, dict(k_out=BASE + 2 * STEP)),                                 # over q_out
    (ERR_ALIAS, dict(k_out=BASE + 6 * STEP)),                                 # over the table
    (ERR_ALIAS, dict(q_out=BASE + 4 * STEP)),                                 # over a weight
])
def test_norm_rope_fwd_refusals(lib, code, change):
    assert rope(lib, False, **change) == code


@pytest.mark.parametrize("code,change", [
    (ERR_NULL, dict(dq=0)),
    (ERR_NULL, dict(dk_out=0)),
    (ERR_NULL, dict(work=0)),
    (ERR_NULL, dict(work=0, dqw=0)),
    (ERR_ALIGN, dict(work=BASE + 20 * STEP + 8)),
    (ERR_ALIGN, dict(dqw=BASE + 20 * STEP + 2)),
    (ERR_ALIAS, dict(dq=BASE + STEP)),                                        # over k
    (ERR_ALIAS, dict(dq=BASE + 3 * STEP)),                                    # over k's gradient
    (ERR_ALIAS, dict(dq=BASE + 5 * STEP)),                                    # over dk
    (ERR_ALIAS, dict(dqw=BASE + 7 * STEP)),                                   # over the other weight's
    (ERR_ALIAS, dict(dqw=BASE + 8 * STEP)),                                   # over the weight
    (ERR_ALIAS, dict(work=BASE)),
    (ERR_ALIAS, dict(work=BASE + 4 * STEP)),
    (ERR_ALIAS, dict(work=BASE + 10 * STEP)),
    (ERR_UNSUPPORTED, dict(norm=0, q_weight=0, k_weight=0)),                  # gradients of weights without the norm
    (ERR_UNSUPPORTED, dict(dims=(1, 4, 8, 16, 2, 0, 32), k=0, dk_out=0, dk=0, k_weight=0)),   # ... or without k
])
def test_norm_rope_bwd_refusals(lib, code, change):
    assert rope(lib, True, **change) == code


def test_calls_that_are_taken(lib):
    """In place, blocks of one fused tensor, q alone, no rotation: they pass every
    check and then fail for want of a GPU."""
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    fused = dict(q=BASE, k=BASE + 128, q_out=BASE, k_out=BASE + 128, strides=(192,) * 4)
    alone = dict(dims=(1, 4, 8, 16, 2, 0, 32), k=0, k_weight=0)
    for change in ({}, fused, dict(q_out=BASE), dict(alone, k_out=0), dict(table=0, turned=(0, 0, 0)),
                   dict(norm=0, q_eps=0.0, k_eps=0.0, q_weight=0, k_weight=0)):
        assert rope(lib, False, **change) == ERR_CUDA, change
    fused = dict(q=BASE, k=BASE + 128, dq=BASE + 5 * STEP, dk=BASE + 5 * STEP + 128, strides=(192, 192, 64, 64, 192, 192))
    for change in ({}, fused, dict(dq=BASE + 2 * STEP), dict(dk=BASE + STEP), dict(dqw=0, dkw=0, work=0),
                   dict(alone, dk_out=0, dk=0, dkw=0)):
        assert rope(lib, True, **change) == ERR_CUDA, change


@pytest.mark.parametrize("code,change", [
    (ERR_SHAPE, dict(n=(0, 2, 3))),
    (ERR_SHAPE, dict(r=(3, 2, 2))),
    (ERR_SHAPE, dict(r=(0, 0, 0))),
    (ERR_SHAPE, dict(r=(2, -2, 2))),
    (ERR_OVERFLOW, dict(n=(1 << 28, 1, 1), r=(2, 0, 0))),
    (ERR_OVERFLOW, dict(n=(1 << 62, 1, 1))),
    (ERR_UNSUPPORTED, dict(theta=0.0)),
    (ERR_UNSUPPORTED, dict(theta=NAN)),
    (ERR_UNSUPPORTED, dict(offset=(INF, 0, 0))),
    (ERR_UNSUPPORTED, dict(scale=(1, NAN, 1))),
    (ERR_NULL, dict(at=0)),
    (ERR_ALIGN, dict(at=BASE + 4)),
])
def test_rope_table_refusals(lib, code, change):
    o = dict(at=BASE, n=(2, 3, 4), r=(4, 2, 2), theta=10000.0, offset=(0, 0, 0), scale=(1, 1, 1))
    o.update(change)
    assert lib.na3d_rope_table(P(o["at"]), *o["n"], *o["r"], o["theta"], *o["offset"], *o["scale"], None) == code


def cross(lib, backward, sizes=(2, 100, 40, 4, 2, 32), strides=None, doc=BASE + 12 * STEP, kv_doc=BASE + 13 * STEP, **ptrs):
    names = ("q", "k", "v", "out", "lse", "work")
    if backward:
        names = ("q", "k", "v", "out", "lse", "dout", "dq", "dk", "dv", "work")
    at = {n: BASE + i * STEP for i, n in enumerate(names)}
    at.update(ptrs)
    rows = (sizes[3] * sizes[5], sizes[4] * sizes[5], sizes[4] * sizes[5])
    call = lib.na3d_cross_bwd if backward else lib.na3d_cross_fwd
    return call(*[P(at[n]) for n in names], *sizes, *(strides or rows * (2 if backward else 1)), P(doc), P(kv_doc), None)


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("code,change", [
    (ERR_SHAPE, dict(sizes=(0, 100, 40, 4, 2, 32))),
    (ERR_SHAPE, dict(sizes=(2, 0, 40, 4, 2, 32))),
    (ERR_SHAPE, dict(sizes=(2, 100, 0, 4, 2, 32))),
    (ERR_SHAPE, dict(sizes=(2, 100, 40, 4, 3, 32))),
    (ERR_HEAD_DIM, dict(sizes=(2, 100, 40, 4, 2, 24))),
    (ERR_UNSUPPORTED, dict(sizes=(2, 100, 40, 4, 2, 256))),
    (ERR_UNSUPPORTED, dict(sizes=(2, 100, 40, 65, 1, 16))),
    (ERR_OVERFLOW, dict(sizes=(2, 1 << 31, 40, 4, 2, 32))),
    (ERR_OVERFLOW, dict(sizes=(2, 100, 1 << 31, 4, 2, 32))),
    (ERR_OVERFLOW, dict(sizes=(1 << 20, 1 << 20, 40, 4, 2, 32))),
    (ERR_NULL, dict(q=0)),
    (ERR_NULL, dict(v=0)),
    (ERR_NULL, dict(out=0)),
    (ERR_ALIGN, dict(k=BASE + STEP + 8)),
    (ERR_ALIGN, dict(lse=BASE + 4 * STEP + 2)),
    (ERR_ALIGN, dict(doc=BASE + 12 * STEP + 2)),
    (ERR_ALIGN, dict(kv_doc=BASE + 12 * STEP + 1)),
])
def test_cross_refusals(lib, backward, code, change):
    assert cross(lib, backward, **change) == code


@pytest.mark.parametrize("code,change", [
    (ERR_SHAPE, dict(strides=(120, 64, 64))),
    (ERR_SHAPE, dict(strides=(128, 56, 64))),
    (ERR_ALIGN, dict(strides=(128, 64, 68))),
    (ERR_OVERFLOW, dict(strides=(1 << 39, 64, 64))),
    (ERR_ALIAS, dict(out=BASE)),
    (ERR_ALIAS, dict(out=BASE + STEP)),
    (ERR_ALIAS, dict(lse=BASE + 3 * STEP + 64)),
    (ERR_ALIAS, dict(lse=BASE + 12 * STEP)),
    (ERR_ALIAS, dict(out=BASE + 13 * STEP)),
])
def test_cross_fwd_refusals(lib, code, change):
    assert cross(lib, False, **change) == code


@pytest.mark.parametrize("code,change", [
    (ERR_NULL, dict(lse=0)),
    (ERR_NULL, dict(dout=0)),
    (ERR_NULL, dict(dv=0)),
    (ERR_NULL, dict(work=0)),
    (ERR_ALIGN, dict(dout=BASE + 5 * STEP + 8)),
    (ERR_ALIGN, dict(work=BASE + 9 * STEP + 8)),
    (ERR_ALIAS, dict(dq=BASE)),
    (ERR_ALIAS, dict(dk=BASE + 3 * STEP)),
    (ERR_ALIAS, dict(dk=BASE + 6 * STEP)),                                    # over dq
    (ERR_ALIAS, dict(dv=BASE + 7 * STEP + 32)),                               # beside dk
    (ERR_ALIAS, dict(strides=(128, 64, 64, 128, 96, 96), dv=BASE + 7 * STEP + 128)),   # rows that wrap into dk's next
    (ERR_ALIAS, dict(work=BASE + 8 * STEP)),
    (ERR_ALIAS, dict(work=BASE + 5 * STEP)),
    (ERR_ALIAS, dict(work=BASE + 12 * STEP)),
])
def test_cross_bwd_refusals(lib, code, change):
    assert cross(lib, True, **change) == code


def test_cross_takes_fused_blocks(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    kv = dict(k=BASE + STEP, v=BASE + STEP + 128)
    assert cross(lib, False) == ERR_CUDA and cross(lib, False, doc=0, kv_doc=0, lse=0) == ERR_CUDA
    assert cross(lib, False, strides=(128, 128, 128), **kv) == ERR_CUDA
    assert cross(lib, True, strides=(128, 128, 128) * 2, dk=BASE + 7 * STEP, dv=BASE + 7 * STEP + 128, **kv) == ERR_CUDA
    assert lib.na3d_cross_workspace(2, 100, 40, 4, 2, 32, 1) > 0
    assert lib.na3d_cross_workspace(2, 100, 40, 4, 3, 32, 0) == -1
    assert lib.na3d_norm_rope_workspace(128) > 0 and lib.na3d_norm_rope_workspace(96) == -1


def test_binding_refuses_before_the_call():
    """Host tensors, other types and shapes that do not go together."""
    na_build.build()
    q = torch.zeros((1, 2, 3, 4, 2, 32), dtype=torch.bfloat16)
    kv = torch.zeros((1, 5, 2, 32), dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        na.na3d_norm_rope(q, q, q.clone(), q.clone())
    with pytest.raises(TypeError):
        na.na3d_cross_attention(q, kv, kv)
    with pytest.raises(TypeError):
        na.na3d_cross_attention([1], kv, kv)
    with pytest.raises(na.NA3DError):
        na.na3d_rope_table((2, 0, 2), (2, 2, 2))
    with pytest.raises(ValueError):
        na.na3d_norm_rope_workspace(48)
    with pytest.raises(ValueError):
        na.na3d_cross_workspace(1, 10, 10, 4, 3, 64)
