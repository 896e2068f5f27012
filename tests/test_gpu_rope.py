"""The norm and rotation of queries and keys on the GPU against the 64-bit
reference, forward and backward, every value within the derived bound."""
import pytest
import torch

import block_reference as ref
import neighborhood_attention_video_gb300 as na
from packed_reference import check

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def make(shape, NKV, seed, scale=1.0):
    """q, k (and gradients and weights) as views of one fused tensor on the CPU."""
    B, T, H, W, NH, HD = shape
    gen = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=gen).to(BF16)  # noqa: E731
    qkv = (torch.randn((B, T, H, W, NH + 2 * NKV, HD), generator=gen) * scale).to(BF16)
    return qkv, rand(*shape), rand(B, T, H, W, NKV, HD), rand(HD), rand(HD)


CASES = [
    # shape (B,T,H,W,NH,HD), heads of k, values turned, interleaved, norm, weights
    ((1, 1, 1, 1, 1, 16), 1, (4, 4, 4), True, True, True),
    ((1, 2, 3, 5, 2, 16), 1, (0, 0, 0), True, True, True),
    ((2, 3, 4, 5, 3, 16), 3, (6, 6, 4), False, True, True),
    ((2, 6, 5, 7, 6, 32), 3, (8, 12, 8), True, True, True),
    ((1, 5, 9, 3, 4, 32), 4, (8, 4, 4), False, True, False),
    ((1, 4, 6, 10, 8, 64), 8, (16, 24, 24), False, True, True),
    ((3, 2, 7, 9, 5, 64), 1, (20, 22, 22), True, False, False),
    ((2, 1, 1, 1, 16, 128), 16, (44, 42, 42), True, True, True),
    ((1, 3, 8, 11, 9, 128), 3, (0, 64, 64), False, True, True),
    ((1, 2, 5, 6, 33, 128), 0, (128, 0, 0), True, True, True),
    ((1, 2, 4, 4, 3, 128), 2, (16, 16, 0), False, False, False),
    ((1, 2, 3, 4, 2, 256), 1, (80, 80, 96), True, True, True),
    ((2, 2, 3, 2, 3, 512), 2, (200, 100, 100), False, True, True),
    ((1, 16, 24, 30, 2, 64), 2, (20, 22, 22), True, True, True),
    ((1, 1, 1, 700, 1, 16), 1, (0, 0, 16), False, True, True),
]


@pytest.mark.parametrize("shape,NKV,dims,inter,norm,weights", CASES, ids=lambda v: str(v).replace(" ", ""))
def test_matches_the_reference(shape, NKV, dims, inter, norm, weights):
    B, T, H, W, NH, HD = shape
    qkv, gq, gk, wq, wk = make(shape, NKV, sum(shape))
    how = dict(norm=norm, interleaved=inter)
    w = dict(q_weight=wq.cuda() if weights else None, k_weight=wk.cuda() if weights and NKV else None)
    table = na.na3d_rope_table((T, H, W), dims, theta=500.0) if any(dims) else None
    dev = qkv.cuda()
    q, k = dev[..., :NH, :], dev[..., NH:NH + NKV, :] if NKV else None
    out = torch.full((B, T, H, W, NH + NKV, HD), float("nan"), dtype=BF16, device="cuda")
    qo, ko = out[..., :NH, :], out[..., NH:, :] if NKV else None
    args = dict(w, table=table, rope_dims=dims, q_eps=1e-4, k_eps=1e-6, q_scale=HD ** -0.5, **how)
    na.na3d_norm_rope(q, k, qo, ko, **args)
    dq = torch.full_like(gq, float("nan"), device="cuda")
    dk = torch.full_like(gk, float("nan"), device="cuda") if NKV else None
    dw = [torch.full((HD,), float("nan"), device="cuda") if norm and (i == 0 or NKV) else None for i in range(2)]
    na.na3d_norm_rope_bwd(q, k, gq.cuda(), gk.cuda() if NKV else None, dq, dk, dq_weight=dw[0], dk_weight=dw[1], **args)
    torch.cuda.synchronize()
    ang = ref.angles((T, H, W), dims, theta=500.0)
    for name, x, wt, eps, sc, g, got in (("q", qkv[..., :NH, :], wq, 1e-4, HD ** -0.5, gq, (qo, dq, dw[0])),
                                         ("k", qkv[..., NH:NH + NKV, :], wk, 1e-6, 1.0, gk, (ko, dk, dw[1]))):
        if got[0] is None:
            continue
        want = ref.norm_rope(x, ang, wt if weights else None, eps=eps, scale=sc, dout=g, **how)
        check(name, got[0], want["out"])
        check("d" + name, got[1], want["dx"])
        if norm:
            check(name + " weight", got[2], want["dw"])


def test_table():
    """Angles of far, shifted and stretched positions, to a step of fp32."""
    for grid, dims, how in (((3, 5, 7), (4, 2, 6), {}), ((1, 1, 9), (0, 0, 128), dict(theta=1e6)),
                            ((4, 2, 2), (16, 8, 8), dict(offset=(1e6, -3.5, 77777.25), scale=(1.0, 0.125, 333.0)))):
        got, want = na.na3d_rope_table(grid, dims, **how).cpu().double(), ref.table(grid, dims, **how)
        # fp32 rounding, and 64-bit angles of up to 2^20 radians
        assert got.shape == want.shape and float((got - want).abs().max()) <= 2.0 ** -25 + 2.0 ** -30


def test_in_place_and_blocks_of_one_tensor():
    """Outputs over their inputs, and gradients over those they come from, equal the others' bits."""
    shape, NKV, dims = (2, 3, 4, 6, 4, 64), 2, (16, 24, 16)
    qkv, gq, gk, wq, wk = (x.cuda() for x in make(shape, NKV, 5))
    NH = shape[4]
    args = dict(q_weight=wq, k_weight=wk, table=na.na3d_rope_table(shape[1:4], dims), rope_dims=dims)
    blocks = lambda t: (t[..., :NH, :], t[..., NH:NH + NKV, :])  # noqa: E731
    a, b = torch.empty_like(gq), torch.empty_like(gk)
    na.na3d_norm_rope(*blocks(qkv), a, b, **args)
    here = qkv.clone()
    na.na3d_norm_rope(*blocks(here), *blocks(here), **args)
    assert torch.equal(blocks(here)[0], a) and torch.equal(blocks(here)[1], b)
    assert torch.equal(here[..., NH + NKV:, :], qkv[..., NH + NKV:, :])
    dq, dk = torch.empty_like(gq), torch.empty_like(gk)
    na.na3d_norm_rope_bwd(*blocks(qkv), gq, gk, dq, dk, **args)
    for over in ("gradient", "input"):
        x, g, h = qkv.clone(), gq.clone(), gk.clone()
        na.na3d_norm_rope_bwd(*blocks(x), g, h, *((g, h) if over == "gradient" else blocks(x)), **args)
        got = (g, h) if over == "gradient" else blocks(x)
        assert torch.equal(got[0], dq) and torch.equal(got[1], dk)


def test_padding_rows_stay_by_themselves():
    """Rows of NaN and infinity whose gradient is 0 give 0 and leave the weights' gradients alone."""
    shape, NKV, dims = (1, 2, 5, 8, 3, 32), 3, (8, 12, 12)
    qkv, gq, gk, wq, wk = (x.cuda() for x in make(shape, NKV, 6))
    gq[:, :, :, 6:], gk[:, :, :, 6:] = 0, 0
    args = dict(q_weight=wq, k_weight=wk, table=na.na3d_rope_table(shape[1:4], dims), rope_dims=dims)
    results = []
    for fill in (None, float("nan"), float("inf")):
        x = qkv.clone()
        if fill is not None:
            x[:, :, :, 6:] = fill
        q, k = x[..., :3, :], x[..., 3:6, :]
        o = [torch.empty_like(gq) for _ in range(4)] + [torch.empty(32, device="cuda") for _ in range(2)]
        na.na3d_norm_rope(q, k, o[0], o[1], **args)
        na.na3d_norm_rope_bwd(q, k, gq, gk, o[2], o[3], dq_weight=o[4], dk_weight=o[5], **args)
        assert not o[2][:, :, :, 6:].any() and not o[3][:, :, :, 6:].any()
        results.append([t[:, :, :, :6] if t.dim() == 6 else t for t in o])
    for other in results[1:]:
        assert all(torch.equal(a, b) for a, b in zip(results[0], other))


def test_zero_rows_and_large_values():
    """A head of zeros stays 0; values to 2^40 are normed like small ones."""
    shape, dims = (1, 1, 2, 3, 2, 64), (0, 32, 32)
    qkv, gq, gk, wq, wk = make(shape, 2, 7)
    qkv[0, 0, 0, 0] = 0
    qkv[0, 0, 0, 1] *= 2.0 ** 40
    qkv[0, 0, 0, 2] *= 2.0 ** -40
    table = na.na3d_rope_table((1, 2, 3), dims)
    out = torch.empty_like(gq, device="cuda")
    dev = qkv.cuda()
    na.na3d_norm_rope(dev[..., :2, :], None, out, None, q_weight=wq.cuda(), table=table, rope_dims=dims)
    check("q", out, ref.norm_rope(qkv[..., :2, :], ref.angles((1, 2, 3), dims), wq)["out"])
    assert not out[0, 0, 0, 0].any()


def test_graph_streams_and_repeats():
    """A captured pair of calls follows its inputs; two streams at once; equal bits on every run."""
    shape, NKV, dims = (1, 4, 10, 12, 4, 64), 4, (16, 24, 24)
    table = na.na3d_rope_table(shape[1:4], dims)

    def buffers(seed):
        x, gq, gk, wq, wk = (t.cuda() for t in make(shape, NKV, seed))
        o = [torch.empty_like(gq), torch.empty_like(gk), torch.empty_like(gq), torch.empty_like(gk),
             torch.empty(64, device="cuda"), torch.empty(64, device="cuda")]
        return x, gq, gk, wq, wk, o

    def call(x, gq, gk, wq, wk, o):
        args = dict(q_weight=wq, k_weight=wk, table=table, rope_dims=dims)
        q, k = x[..., :4, :], x[..., 4:8, :]
        na.na3d_norm_rope(q, k, o[0], o[1], **args)
        na.na3d_norm_rope_bwd(q, k, gq, gk, o[2], o[3], dq_weight=o[4], dk_weight=o[5], **args)

    want = []
    for seed in (1, 2):
        b = buffers(seed)
        call(*b)
        want.append([t.clone() for t in b[-1]])
    # two streams
    sets, streams = [buffers(s) for s in (1, 2)], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for b, s in zip(sets, streams):
            with torch.cuda.stream(s):
                call(*b)
    torch.cuda.synchronize()
    for b, w in zip(sets, want):
        assert all(torch.equal(x, y) for x, y in zip(b[-1], w))
    # captured on inputs 1, replayed on inputs 2
    b, other = buffers(1), buffers(2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(*b)
    for x, y in zip(b[:5], other[:5]):
        x.copy_(y)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(b[-1], want[1]))


def test_past_32_bits():
    """More than 2^31 values: the last frame's rows are those of the frame by itself."""
    B, T, H, W, NH, HD, dims = 1, 34, 128, 128, 32, 128, (44, 42, 42)
    shape, last = (B, T, H, W, NH, HD), (B, 1, H, W, NH, HD)
    q = torch.empty(shape, dtype=BF16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(5))
    out = torch.empty_like(q)
    table = na.na3d_rope_table((T, H, W), dims)
    na.na3d_norm_rope(q, None, out, None, table=table, rope_dims=dims)
    want = torch.empty(last, dtype=BF16, device="cuda")
    alone = dict(table=na.na3d_rope_table((1, H, W), dims, offset=(T - 1, 0, 0)), rope_dims=dims)
    na.na3d_norm_rope(q[:, -1:], None, want, None, **alone)
    assert torch.equal(out[:, -1:], want)
    dq = torch.empty_like(q)
    na.na3d_norm_rope_bwd(q, None, out, None, dq, None, table=table, rope_dims=dims)
    na.na3d_norm_rope_bwd(q[:, -1:], None, out[:, -1:], None, want, None, **alone)
    assert torch.equal(dq[:, -1:], want)
