"""The 64-bit references of the norm, rotation and cross attention against
autograd, differences and cases known by hand; no GPU needed."""
import math

import pytest
import torch

import block_reference as ref

F64 = torch.float64


def rand(gen, *shape):
    return torch.randn(shape, generator=gen, dtype=F64)


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("norm", [True, False])
def test_norm_rope_gradients_are_differences(interleaved, norm):
    gen = torch.Generator().manual_seed(1)
    grid, dims = (2, 3, 2), (4, 8, 4)
    x, g, w = rand(gen, 1, *grid, 2, 32), rand(gen, 1, *grid, 2, 32), rand(gen, 32)
    ang = ref.angles(grid, dims)
    how = dict(norm=norm, eps=1e-3, scale=0.7, interleaved=interleaved)
    f = lambda x, w: float((ref.norm_rope(x, ang, w if norm else None, **how)["out"][0] * g).sum())  # noqa: E731
    got = ref.norm_rope(x, ang, w if norm else None, dout=g, **how)
    for name, at, h in (("dx", x, 1e-5), ("dw", w, 1e-5)):
        if name not in got:
            continue
        step = rand(gen, *at.shape)
        a, b = ((f(at + s * step, w) if name == "dx" else f(x, at + s * step)) for s in (h, -h))
        assert math.isclose((a - b) / (2 * h), float((got[name][0] * step).sum()), rel_tol=1e-6)


def test_rotation_depends_on_the_distance_alone():
    """The product of a turned q and a turned k is that of the positions' difference,
    and a rotation keeps the length."""
    gen = torch.Generator().manual_seed(2)
    grid, dims = (4, 5, 6), (8, 4, 4)
    q, k = rand(gen, 32).expand(1, *grid, 1, 32), rand(gen, 32).expand(1, *grid, 1, 32)
    ang = ref.angles(grid, dims)
    for inter in (True, False):
        a, b = (ref.norm_rope(x, ang, norm=False, interleaved=inter)["out"][0][0, ..., 0, :] for x in (q, k))
        assert torch.allclose((a[1, 2, 3] * b[0, 1, 1]).sum(), (a[3, 4, 5] * b[2, 3, 3]).sum())
        assert torch.allclose(a.norm(dim=-1), q[0, ..., 0, :].norm(dim=-1))
        assert torch.equal(a[0, 0, 0], q[0, 0, 0, 0, 0])
        assert torch.equal(a[..., 16:], q[0, ..., 0, 16:])


def test_table_layout():
    t = ref.table((2, 3, 4), (4, 2, 0))
    assert t.shape == (2 * 2 + 3 * 1, 2)
    assert torch.allclose(t[3], torch.tensor([math.cos(0.01), math.sin(0.01)], dtype=F64))     # t = 1, second pair
    assert torch.allclose(t[6], torch.tensor([math.cos(2.0), math.sin(2.0)], dtype=F64))       # h = 2


def test_cross_against_autograd():
    gen = torch.Generator().manual_seed(3)
    B, T, H, W, NH, NKV, HD, S = 2, 2, 1, 3, 4, 2, 16, 5
    q, k, v = (rand(gen, *s).requires_grad_() for s in ((B, T, H, W, NH, HD), (B, S, NKV, HD), (B, S, NKV, HD)))
    g = rand(gen, B, T, H, W, NH, HD)
    doc = torch.tensor([[0, 0, 1, 1, -1, 2], [3, 3, 3, 0, 0, 0]], dtype=torch.int32).view(B, T, H, W)
    kv_doc = torch.tensor([[0, 1, 1, 0, -1], [3, 3, 3, 3, 3]], dtype=torch.int32)
    see = (doc.view(B, -1, 1) == kv_doc[:, None]) & (kv_doc >= 0)[:, None]
    s = torch.einsum("blhd,bshd->bhls", q.reshape(B, -1, NH, HD), k.repeat_interleave(2, 2))
    s = s.masked_fill(~see[:, None], -math.inf)
    p = torch.where(see[:, None], torch.softmax(torch.where(see.any(-1)[:, None, :, None], s, 0.0), -1), 0.0)
    out = torch.einsum("bhls,bshd->blhd", p, v.repeat_interleave(2, 2)).reshape(q.shape)
    out.backward(g)
    got = ref.cross(q, k, v, doc, kv_doc, g)
    for name, want in (("out", out), ("dq", q.grad), ("dk", k.grad), ("dv", v.grad)):
        assert torch.allclose(got[name][0], want.detach(), atol=1e-12), name
    assert torch.isinf(got["lse"][0][0, 1, 0, 1]).all() and torch.isinf(got["lse"][0][0, 1, 0, 2]).all()
    assert torch.isinf(got["lse"][0][1, 1]).all()
