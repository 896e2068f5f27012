"""The attention to states of another length on the GPU against the 64-bit
reference, forward and backward, every value within the derived bound."""
import pytest
import torch

import block_reference as ref
import neighborhood_attention_video_gb300 as na
from packed_reference import check

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def make(shape, S, NKV, seed, scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    B, HD = shape[0], shape[5]
    q = (torch.randn(shape, generator=gen) * scale * HD ** -0.5).to(BF16)
    kv = torch.randn((B, S, 2, NKV, HD), generator=gen).to(BF16)
    return q, kv, torch.randn(shape, generator=gen).to(BF16)


def make_docs(shape, S, docs, seed, order="runs"):
    """Documents of tokens and states: runs along T and S, or scattered; one without
    states, one without tokens, padding on both sides."""
    B, T, H, W = shape[:4]
    if not docs:
        return None, None
    gen = torch.Generator().manual_seed(seed + 1)
    L = T * H * W
    if order == "scattered":
        doc = torch.randint(-1, docs, (B, L), generator=gen)
        kv = torch.randint(-1, docs + 1, (B, S), generator=gen)
    else:
        cuts = torch.randint(0, L + 1, (B, docs - 1), generator=gen)
        doc = (torch.arange(L)[None, :, None] >= cuts[:, None]).sum(-1)
        doc[:, L - L // 9:] = -3
        share = -(-S // docs)
        kv = (torch.arange(S) // share).expand(B, S).clone()
        length = torch.randint(0, share + 1, (B, docs), generator=gen)
        kv[(torch.arange(S) % share)[None] >= length.gather(1, kv)] = -1
    return doc.view(B, T, H, W).to(torch.int32), kv.to(torch.int32)


def run(q, kv, g, doc=None, kv_doc=None, stream=None):
    """Forward and backward through fused views; gradients start as NaN."""
    q, kv, g, doc, kv_doc = (None if x is None else x.cuda() for x in (q, kv, g, doc, kv_doc))
    k, v = kv[:, :, 0], kv[:, :, 1]
    out, lse = na.na3d_cross_attention(q, k, v, doc=doc, kv_doc=kv_doc, return_lse=True)
    dq, dkv = torch.full_like(q, float("nan")), torch.full_like(kv, float("nan"))
    na.na3d_cross_bwd(q, k, v, out, lse, g, dq, dkv[:, :, 0], dkv[:, :, 1], doc=doc, kv_doc=kv_doc)
    torch.cuda.synchronize()
    return dict(out=out, lse=lse, dq=dq, dk=dkv[:, :, 0], dv=dkv[:, :, 1])


CASES = [
    # shape (B,T,H,W,NH,HD), states, heads of k and v, documents, their order
    ((1, 1, 1, 1, 1, 16), 1, 1, 0, ""),
    ((1, 1, 1, 1, 1, 128), 1, 1, 0, ""),
    ((1, 1, 1, 3, 2, 64), 2, 2, 0, ""),
    ((2, 1, 1, 1, 8, 128), 300, 8, 0, ""),
    ((3, 1, 1, 1, 16, 64), 515, 4, 2, "runs"),
    ((1, 1, 1, 1, 4, 32), 5000, 1, 0, ""),
    ((1, 1, 1, 2, 6, 128), 4100, 2, 3, "scattered"),
    ((1, 2, 8, 8, 2, 64), 128, 2, 0, ""),
    ((1, 2, 8, 8, 2, 128), 64, 2, 0, ""),
    ((1, 3, 7, 11, 3, 16), 77, 3, 0, ""),
    ((2, 3, 7, 11, 6, 32), 77, 2, 2, "runs"),
    ((2, 4, 9, 10, 4, 64), 200, 4, 3, "runs"),
    ((1, 5, 8, 9, 2, 128), 257, 1, 4, "runs"),
    ((2, 2, 9, 13, 2, 64), 190, 2, 5, "scattered"),
    ((1, 2, 9, 13, 4, 128), 131, 2, 3, "scattered"),
    ((1, 1, 3, 50, 5, 32), 129, 1, 0, ""),
    ((1, 1, 2, 9, 64, 16), 65, 1, 0, ""),
    ((1, 1, 4, 33, 7, 64), 127, 1, 2, "runs"),
    ((4, 1, 5, 5, 2, 64), 640, 2, 0, ""),
    ((1, 9, 10, 13, 1, 128), 383, 1, 0, ""),
    ((1, 1, 1, 600, 2, 16), 600, 2, 1, "runs"),
    # one row tile, whose column tiles go by turns: passes of one, of an odd number, of none
    ((2, 1, 1, 5, 8, 128), 1400, 2, 4, "runs"),
    ((1, 1, 2, 20, 3, 64), 900, 1, 3, "scattered"),
    ((1, 1, 1, 7, 4, 32), 385, 4, 0, ""),
    ((2, 1, 1, 3, 2, 16), 20000, 1, 5, "runs"),
    ((1, 1, 1, 1, 12, 64), 300000, 3, 0, ""),
    # many units of one column tile each to a block
    ((1, 8, 24, 32, 16, 128), 77, 16, 0, ""),
    ((2, 4, 24, 32, 16, 64), 20, 16, 2, "runs"),
]


@pytest.mark.parametrize("shape,S,NKV,docs,order", CASES, ids=lambda v: str(v).replace(" ", ""))
def test_matches_the_reference(shape, S, NKV, docs, order):
    q, kv, g = make(shape, S, NKV, sum(shape) + S)
    doc, kv_doc = make_docs(shape, S, docs, S, order)
    want = ref.cross(q, kv[:, :, 0], kv[:, :, 1], doc, kv_doc, g)
    got = run(q, kv, g, doc, kv_doc)
    for name in want:
        check(name, got[name], want[name])


@pytest.mark.parametrize("scale", [0.0, 1e-3, 10.0, 100.0])
@pytest.mark.parametrize("HD", [32, 128])
def test_large_and_small_scores(scale, HD):
    """Scores far from 0, and rising and falling along the states, keep their softmax."""
    shape, S = (1, 2, 6, 12, 2, HD), 700
    q, kv, g = make(shape, S, 2, 3, scale)
    ramp = torch.linspace(0, 1, S)
    kv[0, :, 0, 0] = (kv[0, :, 0, 0].float() * ramp[:, None]).to(BF16)
    kv[0, :, 0, 1] = (kv[0, :, 0, 1].float() * ramp.flip(0)[:, None]).to(BF16)
    want = ref.cross(q, kv[:, :, 0], kv[:, :, 1], dout=g)
    got = run(q, kv, g)
    for name in want:
        check(name, got[name], want[name])


def test_one_mask_only():
    """Either of doc and kv_doc by itself: the other is document 0."""
    shape, S = (2, 2, 5, 9, 2, 64), 150
    q, kv, g = make(shape, S, 2, 11)
    doc, kv_doc = make_docs(shape, S, 2, 11)
    for a, b in ((doc, None), (None, kv_doc)):
        want = ref.cross(q, kv[:, :, 0], kv[:, :, 1], a, b, g)
        got = run(q, kv, g, a, b)
        for name in want:
            check(name, got[name], want[name])


def test_extreme_documents():
    shape, S = (1, 1, 4, 40, 2, 32), 90
    q, kv, g = make(shape, S, 1, 12)
    doc = torch.full(shape[:4], 2 ** 31 - 1, dtype=torch.int32)
    doc[0, 0, 1], doc[0, 0, 2, ::2], doc[0, 0, 3] = 0, -2 ** 31, 1 << 30
    kv_doc = torch.full((1, S), 2 ** 31 - 1, dtype=torch.int32)
    kv_doc[0, 10:30], kv_doc[0, 30:50:3], kv_doc[0, 80:] = 0, -2 ** 31, 1 << 30
    want = ref.cross(q, kv[:, :, 0], kv[:, :, 1], doc, kv_doc, g)
    got = run(q, kv, g, doc, kv_doc)
    for name in want:
        check(name, got[name], want[name])


def test_nothing_seen_anywhere():
    """No state of any token's document: zeros, -inf, zero gradients."""
    shape, S = (2, 1, 3, 50, 2, 64), 70
    q, kv, g = make(shape, S, 2, 13)
    for kv_doc in (torch.full((2, S), -1, dtype=torch.int32), torch.full((2, S), 5, dtype=torch.int32)):
        got = run(q, kv, g, None, kv_doc)
        assert not got["out"].any() and torch.isneginf(got["lse"]).all()
        assert not got["dq"].any() and not got["dk"].any() and not got["dv"].any()


@pytest.mark.parametrize("HD", [16, 64, 128])
@pytest.mark.parametrize("fill", [float("nan"), float("inf"), -float("inf"), 3.3e38])
@pytest.mark.parametrize("order", ["runs", "scattered"])
def test_unseen_values_reach_nothing(order, fill, HD):
    """Padding, and the states and tokens of one document, hold values that are not
    finite: the other documents keep their bits."""
    shape, S = (1, 2, 9, 13, 4, HD), 190
    q, kv, g = make(shape, S, 2, 14)
    doc, kv_doc = make_docs(shape, S, 3, 14, order)
    clean = run(q, kv, g, doc, kv_doc)
    sick, kv_sick = (doc < 0) | (doc == 1), (kv_doc < 0) | (kv_doc == 1)
    q2, kv2, g2 = q.clone(), kv.clone(), g.clone()
    q2[sick], kv2[kv_sick], g2[sick] = fill, fill, fill
    got = run(q2, kv2, g2, doc, kv_doc)
    for name in ("out", "lse", "dq"):
        assert torch.equal(got[name][~sick], clean[name][~sick]), name
    for name in ("dk", "dv"):
        assert torch.equal(got[name][~kv_sick], clean[name][~kv_sick]), name
    pad, kv_pad = doc < 0, kv_doc < 0
    assert not got["out"][pad].any() and not got["dq"][pad].any() and torch.isneginf(got["lse"][pad]).all()
    assert not got["dk"][kv_pad].any() and not got["dv"][kv_pad].any()


def test_strided_views_and_bounds():
    """q inside a wider tensor, k and v with different strides, gradients inside larger
    buffers whose other values stay."""
    shape, S, NKV = (2, 2, 5, 7, 4, 32), 100, 2
    q, kv, g = make(shape, S, NKV, 15)
    want = ref.cross(q, kv[:, :, 0], kv[:, :, 1], dout=g)
    wide = torch.full((2, 2, 5, 7, 7, 32), float("nan"), dtype=BF16, device="cuda")
    wide[..., 2:6, :] = q.cuda()
    qs = wide[..., 2:6, :]
    ks = torch.full((2, S, 3, 32), float("nan"), dtype=BF16, device="cuda")
    ks[:, :, 1:] = kv[:, :, 0].cuda()
    vs = torch.full((2, S, 5, 32), float("nan"), dtype=BF16, device="cuda")
    vs[:, :, 2:4] = kv[:, :, 1].cuda()
    k, v = ks[:, :, 1:], vs[:, :, 2:4]
    out, lse = na.na3d_cross_attention(qs, k, v, return_lse=True)
    dw, dkw = torch.full_like(wide, 7.0), torch.full((2, S, 6, 32), 7.0, dtype=BF16, device="cuda")
    na.na3d_cross_bwd(qs, k, v, out, lse, g.cuda(), dw[..., 1:5, :], dkw[:, :, 1:3], dkw[:, :, 3:5])
    got = dict(out=out, lse=lse, dq=dw[..., 1:5, :], dk=dkw[:, :, 1:3], dv=dkw[:, :, 3:5])
    for name in want:
        check(name, got[name], want[name])
    assert (dw[..., :1, :] == 7).all() and (dw[..., 5:, :] == 7).all()
    assert (dkw[:, :, :1] == 7).all() and (dkw[:, :, 5:] == 7).all()


def test_entry_by_entry():
    """An entry of a batch equals the entry by itself."""
    shape, S = (3, 1, 6, 20, 4, 64), 130
    q, kv, g = make(shape, S, 2, 16)
    doc, kv_doc = make_docs(shape, S, 2, 16)
    both = run(q, kv, g, doc, kv_doc)
    for b in range(3):
        one = run(*(x[b:b + 1].contiguous() for x in (q, kv, g, doc, kv_doc)))
        for name in ("out", "lse"):
            assert torch.allclose(one[name][0].float(), both[name][b].float(), rtol=2 ** -7, atol=1e-2), name


def test_repeats_have_equal_bits():
    for shape, S, NKV in (((1, 4, 16, 16, 4, 64), 300, 2), ((1, 1, 1, 1, 8, 128), 9000, 2), ((2, 2, 9, 13, 2, 128), 640, 2)):
        q, kv, g = make(shape, S, NKV, 17)
        doc, kv_doc = make_docs(shape, S, 2, 17)
        first = run(q, kv, g, doc, kv_doc)
        for _ in range(5):
            again = run(q, kv, g, doc, kv_doc)
            assert all(torch.equal(first[n], again[n]) for n in first)


@pytest.mark.parametrize("L,S,NH,NKV", [(1, 40000, 16, 4), (300, 1300, 3, 3)])
def test_long_runs_of_lone_row_tiles(L, S, NH, NKV):
    """Blocks whose second row tile is empty, in some units or all, walk many column
    tiles: over thousands of calls, which the operands reach in any order, the bits stay."""
    q, kv, _ = make((5, 1, 1, L, NH, 128), S, NKV, 21)
    q, kv = q.cuda(), kv.cuda()
    first, lse = na.na3d_cross_attention(q, kv[:, :, 0], kv[:, :, 1], return_lse=True)
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(3000):
        out, other = na.na3d_cross_attention(q, kv[:, :, 0], kv[:, :, 1], return_lse=True)
        differ += (out.view(torch.int16) != first.view(torch.int16)).sum() + (other != lse).sum()
    assert int(differ) == 0 and na.na3d_device_status() == 0


def test_two_streams_at_once():
    cases = [((1, 3, 10, 17, 4, 64), 250, 2), ((1, 1, 1, 1, 8, 128), 6000, 2)]
    data = [make(*c, seed) for seed, c in enumerate(cases)]
    want = [run(*x) for x in data]
    sets = [[t.cuda() for t in x] for x in data]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        got = []
        for (q, kv, g), s in zip(sets, streams):
            with torch.cuda.stream(s):
                out, lse = na.na3d_cross_attention(q, kv[:, :, 0], kv[:, :, 1], return_lse=True)
                dq, dkv = torch.empty_like(q), torch.empty_like(kv)
                na.na3d_cross_bwd(q, kv[:, :, 0], kv[:, :, 1], out, lse, g, dq, dkv[:, :, 0], dkv[:, :, 1])
                got.append(dict(out=out, lse=lse, dq=dq, dk=dkv[:, :, 0], dv=dkv[:, :, 1]))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(a[n], b[n]) for n in a)


def test_graph_capture_and_replay():
    """Two captured calls follow new inputs and new documents, also replayed together."""
    shape, S, NKV = (1, 2, 8, 9, 4, 64), 300, 2
    a, b = (make(shape, S, NKV, s) + make_docs(shape, S, 3, s) for s in (21, 22))
    want = run(*b)
    graphs = []
    for case in range(2):
        q, kv, g, doc, kv_doc = (x.cuda() for x in a)
        dq, dkv = torch.empty_like(q), torch.empty_like(kv)
        out, lse = torch.empty_like(q), torch.empty(q.shape[:5], device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            na.na3d_cross_fwd(q, kv[:, :, 0], kv[:, :, 1], out, lse, doc, kv_doc)
            na.na3d_cross_bwd(q, kv[:, :, 0], kv[:, :, 1], out, lse, g, dq, dkv[:, :, 0], dkv[:, :, 1], doc, kv_doc)
        for x, y in zip((q, kv, g, doc, kv_doc), b):
            x.copy_(y)
        graphs.append((graph, torch.cuda.Stream(), dict(out=out, lse=lse, dq=dq, dk=dkv[:, :, 0], dv=dkv[:, :, 1]), (q, kv, g, doc, kv_doc)))
    torch.cuda.synchronize()
    for graph, stream, _, _ in graphs:
        with torch.cuda.stream(stream):
            graph.replay()
    torch.cuda.synchronize()
    for _, _, got, _ in graphs:
        assert all(torch.equal(got[n], want[n]) for n in want)


def test_work_of_the_callers():
    """A workspace of the caller's gives the same bits; one too small is refused."""
    shape, S, NKV = (1, 1, 1, 1, 8, 128), 9000, 2
    q, kv, g = (x.cuda() for x in make(shape, S, NKV, 23))
    k, v = kv[:, :, 0], kv[:, :, 1]
    want = run(q, kv, g)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:5], device="cuda")
    dq, dkv = torch.empty_like(q), torch.empty_like(kv)
    need = [na.na3d_cross_workspace(1, 1, S, 8, NKV, 128, b) for b in (False, True)]
    work = torch.full((max(need) + 64,), 255, dtype=torch.uint8, device="cuda")
    na.na3d_cross_fwd(q, k, v, out, lse, work=work)
    na.na3d_cross_bwd(q, k, v, out, lse, g, dq, dkv[:, :, 0], dkv[:, :, 1], work=work)
    torch.cuda.synchronize()
    assert torch.equal(out, want["out"]) and torch.equal(dq, want["dq"]) and torch.equal(dkv[:, :, 0], want["dk"])
    assert (work[max(need):] == 255).all()
    with pytest.raises(ValueError):
        na.na3d_cross_bwd(q, k, v, out, lse, g, dq, dkv[:, :, 0], dkv[:, :, 1], work=work[:16])


def test_gradients_are_differences():
    """The gradient along a direction against differences of the forward pass in 64 bits."""
    shape, S = (1, 1, 4, 9, 2, 32), 50
    q, kv, g = make(shape, S, 1, 24)
    got = run(q, kv, g)
    gen = torch.Generator().manual_seed(1)
    f = lambda q, kv: float((ref.cross(q, kv[:, :, 0], kv[:, :, 1])["out"][0] * g.double()).sum())  # noqa: E731
    for name, x, grad in (("q", q, got["dq"]), ("kv", kv, torch.stack([got["dk"], got["dv"]], 2))):
        step = torch.randn(x.shape, generator=gen).double()
        h = 1e-5
        at = [(x.double() + s * step) for s in (h, -h)]
        hi, lo = ((f(a, kv.double()) if name == "q" else f(q.double(), a)) for a in at)
        want, have = (hi - lo) / (2 * h), float((grad.cpu().double() * step).sum())
        # every term of the sum is off by a few roundings: 4 half steps of its magnitude, in quadrature
        scale = float((grad.cpu().double() * step).norm())
        assert abs(want - have) <= 4 * 2.0 ** -8 * scale * 4, (name, want, have)


def test_states_past_32_bits():
    """A memory of more than 2^31 values: its last states alone are seen."""
    S, n, NH, HD = 140000, 300, 64, 128
    gen = torch.Generator("cuda").manual_seed(31)
    kv = torch.empty((1, S, 2, NH, HD), dtype=BF16, device="cuda").normal_(generator=gen)
    q, _, g = make((1, 1, 1, 2, NH, HD), 1, 1, 31)
    kv_doc = torch.full((1, S), -1, dtype=torch.int32)
    kv_doc[:, -n:] = 0
    assert kv.numel() > 2 ** 31
    end = kv[:, -n:].cpu()
    want = ref.cross(q, end[:, :, 0], end[:, :, 1], dout=g)
    k, v, q, g, kv_doc = kv[:, :, 0], kv[:, :, 1], q.cuda(), g.cuda(), kv_doc.cuda()
    out, lse = na.na3d_cross_attention(q, k, v, kv_doc=kv_doc, return_lse=True)
    dq, dkv = torch.empty_like(q), torch.full_like(kv, float("nan"))
    na.na3d_cross_bwd(q, k, v, out, lse, g, dq, dkv[:, :, 0], dkv[:, :, 1], kv_doc=kv_doc)
    got = dict(out=out, lse=lse, dq=dq, dk=dkv[:, -n:, 0], dv=dkv[:, -n:, 1])
    for name in want:
        check(name, got[name], want[name])
    assert not dkv[:, :-n].any()


def test_tokens_past_32_bits():
    """More than 2^31 values of q: the last tokens are those of the tokens by themselves."""
    L, n, S, NH, HD = 1100000, 300, 40, 16, 128
    gen = torch.Generator("cuda").manual_seed(32)
    q = torch.empty((1, 1, 1, L, NH, HD), dtype=BF16, device="cuda").normal_(std=HD ** -0.5, generator=gen)
    _, kv, g = make((1, 1, 1, n, NH, HD), S, NH, 32)
    assert q.numel() > 2 ** 31
    want = ref.cross(q[:, :, :, -n:].cpu(), kv[:, :, 0], kv[:, :, 1], dout=g)
    kv = kv.cuda()
    k, v = kv[:, :, 0], kv[:, :, 1]
    out, lse = na.na3d_cross_attention(q, k, v, return_lse=True)
    dout, dq, dkv = torch.zeros_like(q), torch.empty_like(q), torch.empty_like(kv)
    dout[:, :, :, -n:] = g.cuda()
    na.na3d_cross_bwd(q, k, v, out, lse, dout, dq, dkv[:, :, 0], dkv[:, :, 1])
    got = dict(out=out[:, :, :, -n:], lse=lse[:, :, :, -n:], dq=dq[:, :, :, -n:], dk=dkv[:, :, 0], dv=dkv[:, :, 1])
    for name in want:
        check(name, got[name], want[name])
    assert not dq[:, :, :, :-n].any()
