"""The score-shaped attention on the GPU against the 64-bit reference, forward
and backward, every value within the bound that the reference derives."""
import pytest
import torch

import neighborhood_attention_video_gb300 as na
import packed_reference as ref

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def make(shape, seed, scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    q, k, v, g = (torch.randn(shape, generator=gen) for _ in range(4))
    return [(x * s).to(BF16) for x, s in ((q, scale * shape[-1] ** -0.5), (k, 1), (v, 1), (g, 1))]


def make_options(shape, seed, softcap=0.0, slopes=False, docs=0, pad=0, prefix=None):
    B, T, H, W, NH, _ = shape
    gen = torch.Generator().manual_seed(seed + 1000)
    o = dict(softcap=softcap, slopes=None, doc=None, prefix=None)
    if slopes:
        o["slopes"] = torch.rand((NH, 3), generator=gen)
    if docs:
        cuts = torch.randint(0, T + 1, (B, docs - 1), generator=gen)
        doc = (torch.arange(T)[None, :, None] >= cuts[:, None]).sum(-1)[:, :, None, None]
        doc = doc + 7 * torch.randint(0, 2, (B, 1, H, 1), generator=gen)      # and along H
        o["doc"] = doc.expand(B, T, H, W).to(torch.int32).contiguous()
        if pad:
            o["doc"][..., W - pad:] = -1 - torch.arange(pad, dtype=torch.int32)
    if prefix is not None:
        o["prefix"] = torch.tensor([(prefix + b) for b in range(B)], dtype=torch.int32)
    return o


def cuda(o):
    return {n: x.cuda() if isinstance(x, torch.Tensor) else x for n, x in o.items()}


def run(q, k, v, g, kernel, opts):
    """Forward and backward on the GPU through a fused projection's views."""
    o = cuda(opts)
    qkv = torch.stack([q, k, v], 4).cuda()
    views = na.qkv_views(qkv)
    out, lse = na.na3d_scored_attention(*views, kernel, return_lse=True, **o)
    dqkv = torch.full_like(qkv, float("nan"))
    na.na3d_scored_bwd(*views, out, lse, g.cuda(), *na.qkv_views(dqkv), kernel, **o)
    torch.cuda.synchronize()
    return dict(out=out, lse=lse, **dict(zip(("dq", "dk", "dv"), na.qkv_views(dqkv))))


CASES = [
    # shape (B,T,H,W,NH,HD), window, options
    ((1, 4, 8, 16, 2, 32), (3, 5, 5), {}),
    ((1, 1, 1, 1, 1, 16), (1, 1, 1), dict(softcap=5.0, slopes=True)),
    ((1, 3, 9, 13, 2, 64), (1, 1, 1), dict(slopes=True)),
    ((2, 5, 7, 11, 3, 16), (3, 5, 7), dict(softcap=2.0, slopes=True, docs=2, pad=3, prefix=0)),
    ((1, 8, 16, 16, 2, 64), (3, 7, 7), dict(softcap=30.0, slopes=True)),
    ((1, 6, 10, 18, 2, 64), (3, 7, 7), dict(docs=3)),
    ((2, 6, 9, 14, 1, 128), (3, 5, 5), dict(prefix=2)),
    ((1, 5, 12, 10, 2, 128), (5, 3, 7), dict(softcap=1.0, slopes=True, docs=2, pad=1, prefix=1)),
    ((1, 4, 11, 33, 2, 64), (3, 7, 33), dict(slopes=True, docs=2, pad=4)),
    ((1, 1, 1, 70, 2, 32), (1, 1, 45), dict(softcap=10.0, prefix=0)),
    ((1, 40, 1, 1, 2, 32), (21, 1, 1), dict(prefix=3, slopes=True)),
    ((1, 1, 37, 3, 2, 16), (1, 37, 3), dict(docs=1)),
    ((1, 12, 13, 13, 1, 64), (11, 11, 11), dict(softcap=50.0)),
    ((3, 2, 5, 6, 5, 32), (1, 5, 3), dict(docs=2, pad=5)),
    ((1, 2, 3, 200, 1, 64), (1, 3, 151), dict(slopes=True)),
    # windows too wide for a table of biases, with and without what the plain steps leave out
    ((1, 2, 40, 40, 1, 128), (1, 31, 33), dict(softcap=10.0, slopes=True, docs=2, pad=3)),
    ((1, 1, 80, 64, 1, 64), (1, 61, 55), dict()),
    # rows of columns in several chunks
    ((1, 1, 2, 700, 1, 32), (1, 1, 501), dict(slopes=True, docs=1, pad=100)),
    # more frames than a warp's rows, causal
    ((2, 33, 4, 5, 2, 32), (9, 3, 3), dict(softcap=40.0, docs=3, prefix=4)),
]


@pytest.mark.parametrize("shape,kernel,opts", CASES, ids=lambda v: str(v).replace(" ", ""))
def test_matches_the_reference(shape, kernel, opts):
    q, k, v, g = make(shape, sum(shape) + sum(kernel))
    o = make_options(shape, sum(shape), **opts)
    want = ref.scored(q, k, v, kernel, dout=g, **o)
    got = run(q, k, v, g, kernel, o)
    for name in want:
        ref.check(name, got[name], want[name])


@pytest.mark.parametrize("scale,softcap", [(30.0, 0.0), (30.0, 8.0), (200.0, 20.0), (1e-3, 2.0 ** -10), (3.0, 2.0 ** 20)])
def test_large_and_small_scores(scale, softcap):
    """Scores far from 0 keep their softmax; caps at both ends of their range."""
    shape, kernel = (1, 4, 9, 11, 2, 64), (3, 5, 5)
    q, k, v, g = make(shape, 17, scale)
    o = dict(softcap=softcap, slopes=None, doc=None, prefix=None)
    want = ref.scored(q, k, v, kernel, dout=g, **o)
    got = run(q, k, v, g, kernel, o)
    for name in want:
        ref.check(name, got[name], want[name])


@pytest.mark.parametrize("softcap,HD", [(0.0, 64), (12.0, 64), (100.0, 32), (64.0, 128), (70.0, 16)])
def test_slopes_of_either_sign(softcap, HD):
    """A bias that grows with the distance, as large as e^60, beside one that
    falls as fast; caps on both sides of those that need no running maximum."""
    shape, kernel = (1, 5, 10, 13, 3, HD), (3, 7, 9)
    q, k, v, g = make(shape, 23, 4.0)
    o = make_options(shape, 23, softcap, True, 2, 2, 1)
    o["slopes"] = torch.tensor([[6.0, -7.0, -5.0], [-3.0, 8.0, 5.0], [0.0, -0.5, 0.25]])
    want = ref.scored(q, k, v, kernel, dout=g, **o)
    got = run(q, k, v, g, kernel, o)
    for name in want:
        ref.check(name, got[name], want[name])


def test_extreme_documents_and_prefixes():
    """Any negative document is padding, documents reach to 2^31 - 1; prefixes
    below 0 and past the last frame."""
    shape, kernel = (2, 5, 6, 9, 1, 32), (3, 3, 5)
    q, k, v, g = make(shape, 29)
    o = make_options(shape, 29)
    o["doc"] = torch.full(shape[:4], 2 ** 31 - 1, dtype=torch.int32)
    o["doc"][0, :, 3:] = 0
    o["doc"][1, 2] = -2 ** 31
    o["doc"][1, :, :, :2] = -1
    for prefix in ((-5, 99), (0, -2 ** 31), (2 ** 31 - 1, 2)):
        o["prefix"] = torch.tensor(prefix, dtype=torch.int64).to(torch.int32)
        want = ref.scored(q, k, v, kernel, dout=g, **o)
        got = run(q, k, v, g, kernel, o)
        for name in want:
            ref.check(name, got[name], want[name])


def test_two_streams_at_once():
    """Forward and backward on two streams, each with a workspace of its own."""
    shape, kernel = (1, 6, 16, 18, 2, 64), (3, 5, 5)
    data = [(make(shape, s), make_options(shape, s, 20.0, True, 2, 1)) for s in (1, 2)]
    want = [ref.scored(*x[:3], kernel, dout=x[3], **o) for x, o in data]
    streams = [torch.cuda.Stream() for _ in data]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    results = [None, None]
    for _ in range(5):
        for i, (x, o) in enumerate(data):
            with torch.cuda.stream(streams[i]):
                d, co = [y.cuda() for y in x], cuda(o)
                out, lse = na.na3d_scored_attention(*d[:3], kernel, return_lse=True, **co)
                grads = [torch.empty_like(d[0]) for _ in range(3)]
                na.na3d_scored_bwd(*d[:3], out, lse, d[3], *grads, kernel, **co)
                results[i] = (out, lse, *grads)
    torch.cuda.synchronize()
    for w, r in zip(want, results):
        for name, x in zip(("out", "lse", "dq", "dk", "dv"), r):
            ref.check(name, x, w[name])


def test_stream_argument():
    """stream= of another stream than the current one, the backward pass's own
    workspace with it."""
    shape, kernel = (1, 4, 9, 10, 2, 32), (3, 3, 3)
    x = make(shape, 31)
    d = [y.cuda() for y in x]
    grads = [torch.empty_like(d[0]) for _ in range(3)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out, lse = na.na3d_scored_attention(*d[:3], kernel, return_lse=True, stream=side)
    na.na3d_scored_bwd(*d[:3], out, lse, d[3], *grads, kernel, stream=side)
    side.synchronize()
    want = ref.scored(*x[:3], kernel, dout=x[3])
    for name, y in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *grads)):
        ref.check(name, y, want[name])


def test_random_problems():
    """Forty seeded problems over every option."""
    gen = torch.Generator().manual_seed(5)
    pick = lambda *c: c[int(torch.randint(0, len(c), (1,), generator=gen))]  # noqa: E731
    upto = lambda n: 1 + int(torch.randint(0, n, (1,), generator=gen))  # noqa: E731
    for i in range(40):
        shape = (upto(2), upto(7), upto(14), upto(22), upto(3), pick(16, 32, 64, 128))
        kernel = tuple(1 + 2 * ((upto(min(n, m)) - 1) // 2) for n, m in zip(shape[1:4], (5, 9, 17)))
        o = make_options(shape, i, pick(0.0, 4.0, 30.0), pick(True, False), pick(0, 1, 2, 3), upto(shape[3]) - 1,
                         pick(None, 0, 2))
        q, k, v, g = make(shape, i)
        want = ref.scored(q, k, v, kernel, dout=g, **o)
        got = run(q, k, v, g, kernel, o)
        for name in want:
            ref.check(f"problem {i} {shape} {kernel} {name}", got[name], want[name])


@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf"), 3.0e38])
@pytest.mark.parametrize("HD", [32, 128])
def test_masked_values_reach_nothing(what, HD):
    """Padding, and another clip's keys and queries, may hold anything: rows that
    do not see them keep the bits they have without it."""
    shape, kernel = (1, 6, 8, 12, 2, HD), (3, 5, 5)
    q, k, v, g = make(shape, 3)
    o = make_options(shape, 3)
    o["doc"] = torch.zeros(shape[:4], dtype=torch.int32)
    o["doc"][:, 3:] = 1
    o["doc"][:, :, :, 10:] = -1
    o["softcap"] = 20.0
    clean = {n: x.clone() for n, x in run(q, k, v, g, kernel, o).items()}
    bad = o["doc"] == 1
    bad[:, :, :, 10:] = True
    for x in (q, k, v, g):
        x[bad] = what
    got = run(q, k, v, g, kernel, o)
    keep = o["doc"] == 0
    want = ref.scored(*[torch.where(bad[..., None, None], 0.0, x.float()) for x in (q, k, v)], kernel, dout=torch.where(
        bad[..., None, None], 0.0, g.float()), **o)
    for name in got:
        value, bound = want[name]
        ref.check(name, got[name].cpu()[keep], (value[keep], bound[keep]))
        assert torch.isfinite(clean[name].cpu()[keep]).all()
    pad = (o["doc"] < 0)
    for name in ("out", "dq", "dk", "dv"):
        assert bool((got[name].cpu()[pad] == 0).all()), name
    assert bool(torch.isneginf(got["lse"].cpu()[pad]).all())


@pytest.mark.parametrize("what", [float("nan"), float("inf")])
def test_a_bad_value_stays_in_its_windows(what):
    """A non-finite key or value reaches exactly the queries whose windows hold it."""
    shape, kernel = (1, 5, 9, 20, 1, 64), (3, 3, 5)
    q, k, v, g = make(shape, 4)
    v[0, 2, 4, 9, 0, 5] = what
    got = run(q, k, v, g, kernel, make_options(shape, 4))
    idx = ref.window_index(5, 9, 20, kernel)
    hit = (idx == (2 * 9 + 4) * 20 + 9).any(-1).reshape(5, 9, 20)
    bad = ~torch.isfinite(got["out"].cpu()[0]).all(-1).all(-1)
    assert torch.equal(bad, hit)
    assert torch.isfinite(got["lse"]).all()


def test_same_inputs_same_bits():
    shape, kernel = (1, 6, 16, 17, 4, 64), (3, 5, 7)
    q, k, v, g = make(shape, 8)
    o = make_options(shape, 8, 20.0, True, 2, 2, 1)
    first = {n: x.clone() for n, x in run(q, k, v, g, kernel, o).items()}
    for _ in range(10):
        got = run(q, k, v, g, kernel, o)
        for n in first:
            assert torch.equal(got[n].view(torch.int16 if n != "lse" else torch.int32),
                               first[n].view(torch.int16 if n != "lse" else torch.int32)), n


def test_outputs_stay_inside_their_tensors():
    shape, kernel = (1, 3, 7, 9, 2, 32), (3, 5, 5)
    q, k, v, g = (x.cuda() for x in make(shape, 9))
    n, rows = q.numel(), q.numel() // 32

    def guarded(count, dtype):
        buf = torch.full((count + 256,), 3.0, dtype=dtype, device="cuda")
        return buf, buf[128:128 + count]

    bufs = [guarded(n, BF16) for _ in range(4)] + [guarded(rows, torch.float32)]
    out, dq, dk, dv = (b[1].view(shape) for b in bufs[:4])
    lse = bufs[4][1].view(shape[:5])
    na.na3d_scored_fwd(q, k, v, out, kernel, lse)
    na.na3d_scored_bwd(q, k, v, out, lse, g, dq, dk, dv, kernel)
    torch.cuda.synchronize()
    for buf, view in bufs:
        assert bool((buf[:128] == 3.0).all()) and bool((buf[128 + view.numel():] == 3.0).all())


def test_streams_and_graph():
    """A call on a side stream, and forward and backward captured into a graph and
    replayed on other inputs, documents included."""
    shape, kernel = (1, 4, 10, 12, 2, 64), (3, 5, 5)
    o = make_options(shape, 1, 20.0, True, 2, 2, 1)
    q, k, v, g = make(shape, 1)
    dev = [x.cuda() for x in (q, k, v, g)]
    co = cuda(o)
    out = torch.empty_like(dev[0])
    lse = torch.empty(shape[:5], device="cuda")
    grads = [torch.empty_like(dev[0]) for _ in range(3)]
    work = torch.empty(na.na3d_scored_bwd_workspace(*shape[:5]), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    side_out = na.na3d_scored_attention(*dev[:3], kernel, stream=side, **co)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        na.na3d_scored_fwd(*dev[:3], out, kernel, lse, **co)
        na.na3d_scored_bwd(*dev[:3], out, lse, dev[3], *grads, kernel, work=work, **co)
    for seed in (1, 2):
        new = make(shape, seed)
        no = make_options(shape, seed, 20.0, True, 2, 2, 1)
        for d, s in zip(dev, new):
            d.copy_(s)
        for name in ("slopes", "doc", "prefix"):
            co[name].copy_(no[name])
        graph.replay()
        torch.cuda.synchronize()
        want = ref.scored(*new[:3], kernel, dout=new[3], **no)
        for name, x in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *grads)):
            ref.check(name, x, want[name])
        if seed == 1:
            assert torch.equal(out, side_out)


def test_offsets_past_32_bits():
    """A fused tensor of more than 2^31 elements: its last rows against the
    reference on their own frames."""
    B, T, H, W, NH, HD = 1, 96, 96, 96, 16, 64
    kernel = (1, 3, 3)
    gen = torch.Generator(device="cuda").manual_seed(3)
    qkv = torch.empty((B, T, H, W, 3, NH, HD), dtype=BF16, device="cuda")
    assert qkv.numel() > 2 ** 31
    for t in range(T):
        qkv[:, t] = torch.randn(qkv[:, t].shape, generator=gen, device="cuda").to(BF16)
    out, lse = na.na3d_scored_attention(*na.qkv_views(qkv), kernel, return_lse=True)
    dqkv = torch.empty_like(qkv)
    na.na3d_scored_bwd(*na.qkv_views(qkv), out, lse, out, *na.qkv_views(dqkv), kernel)
    # frames are independent (KT = 1): the last frame's last rows, whose windows end in row H - 1
    rows = slice(H - 6, H)
    cut = qkv[:, -1:, rows].cpu()
    want = ref.scored(*na.qkv_views(cut), (1, 3, 3), dout=out[:, -1:, rows].cpu())
    for name, x in (("out", out), ("lse", lse), ("dq", na.qkv_views(dqkv)[0])):
        # the first row of the cut has its window elsewhere; the second row's stays
        value, bound = want[name]
        ref.check(name, x[:, -1:, rows].cpu()[:, :, 1:], (value[:, :, 1:], bound[:, :, 1:]))
    for name, x in zip(("dk", "dv"), na.qkv_views(dqkv)[1:]):
        value, bound = want[name]
        ref.check(name, x[:, -1:, rows].cpu()[:, :, 3:], (value[:, :, 3:], bound[:, :, 3:]))


def test_rows_by_themselves_outlast_no_wait():
    """Rows that are not finite are computed one by one, here for longer than the two
    seconds that a wait of the other warps allows: these get their results all the same.
    (Every row of dk and dv sees the bad queries where every window is the whole grid, so
    the bad values enter the backward pass through delta, which only dq takes.)"""
    T, H, W = 41, 91, 99
    shape, kernel = (1, T, H, W, 1, 16), (T, H, W)
    q, k, v, g = (x.cuda() for x in make(shape, 41))
    good = torch.ones(shape[:4], dtype=torch.bool, device="cuda")
    good[:, 0, :4, :4] = False                                    # the rows of one warp
    out, lse = na.na3d_scored_attention(q, k, v, kernel, return_lse=True)
    dq, dk, dv = (torch.empty_like(q) for _ in range(3))
    na.na3d_scored_bwd(q, k, v, out, lse, g, dq, dk, dv, kernel)
    assert na.na3d_device_status() == 0

    q2, out2, lse2 = q.clone(), torch.full_like(out, 7.0), torch.full_like(lse, 7.0)
    q2[~good] = float("nan")
    na.na3d_scored_fwd(q2, k, v, out2, kernel, lse2)
    assert na.na3d_device_status() == 0
    assert torch.equal(out2[good], out[good]) and torch.equal(lse2[good], lse[good])
    assert bool(torch.isnan(out2[~good]).all())

    bad_out = out.clone()
    bad_out[~good] = float("nan")
    dq2, dk2, dv2 = (torch.full_like(q, 7.0) for _ in range(3))
    na.na3d_scored_bwd(q, k, v, bad_out, lse, g, dq2, dk2, dv2, kernel)
    assert na.na3d_device_status() == 0
    assert torch.equal(dq2[good], dq[good]) and bool(torch.isnan(dq2[~good]).all())
    assert bool(torch.isfinite(dk2).all()) and bool(torch.isfinite(dv2).all())


def test_views_of_one_column():
    """A grid cut to one row and column: its frames lie further apart than the strides of
    the axes of one position say."""
    full = torch.stack(make((1, 7, 1, 5, 2, 32), 47)[:3], 4).cuda()
    q, k, v = na.qkv_views(full[:, :, :, :1])
    for opts in ({}, {"doc": torch.zeros((1, 7, 1, 1), dtype=torch.int32, device="cuda")}):
        out = na.na3d_scored_attention(q, k, v, (5, 1, 1), **opts)
        assert torch.equal(out, na.na3d_scored_attention(q.contiguous(), k.contiguous(), v.contiguous(), (5, 1, 1), **opts))
    base = torch.empty_like(out)
    na.na3d_fwd_strided(q, k, v, base, (5, 1, 1))
    assert torch.equal(base, na.na3d_attention(q.contiguous(), k.contiguous(), v.contiguous(), (5, 1, 1)))


@pytest.mark.parametrize("case", range(4))
def test_wide_windows_by_norm(case):
    """Gradients over thousands of keys, whose elementwise bounds would pass a missing
    term: the norm of each result's error against the roundings' expected one."""
    import packed_norms as norms
    from test_packed_norms import WIDE, make as make_wide, slopes_of
    shape, kernel, scale, softcap, slopes = WIDE[case]
    q, k, v, g = make_wide(shape, sum(shape), scale)
    o = dict(softcap=softcap, slopes=slopes_of(shape, slopes), doc=None, prefix=None)
    want = norms.scored(q, k, v, g, kernel, **o)
    got = run(q, k, v, g, kernel, o)
    for name in want:
        assert norms.excess(got[name], want[name]) <= 1, (name, norms.excess(got[name], want[name]))


def test_packed_clips_equal_clips_alone_away_from_cuts():
    """Rows farther than half a window from another clip are those of the clip by itself;
    the rows at a cut see the keys on their side only."""
    shape, kernel, cut = (1, 13, 9, 10, 2, 32), (5, 3, 5), 7
    q, k, v, g = make(shape, 53)
    o = make_options(shape, 53, 15.0, True)
    o["doc"] = (torch.arange(13) >= cut).to(torch.int32)[None, :, None, None].expand(shape[:4]).contiguous()
    got = run(q, k, v, g, kernel, o)
    whole = ref.scored(q, k, v, kernel, **o)
    for frames, away in ((slice(0, cut), slice(0, cut - 2)), (slice(cut, 13), slice(2, 13 - cut))):
        alone = ref.scored(*(x[:, frames] for x in (q, k, v)), kernel, **dict(o, doc=None))
        for name in ("out", "lse"):
            value, bound = alone[name]
            ref.check(name, got[name][:, frames][:, away], (value[:, away], bound[:, away]))
    near = slice(cut - 2, cut + 2)
    for name in ("out", "lse"):
        ref.check(name, got[name][:, near], tuple(x[:, near] for x in whole[name]))


@pytest.mark.parametrize("softcap", [0.5, 8.0, 30.0, 66.0, 67.0, 500.0])
@pytest.mark.parametrize("scale", [0.01, 0.3])
def test_lse_of_small_scores_under_a_cap(softcap, scale):
    """Caps are exact to 2^-21 of the cap: half the exponential's 2^-22, 2^-24 of its sum
    with 1 and 2^-23 of the reciprocal, of a quotient near 1/2 that is taken twice the
    cap times, and the rounding of the score."""
    shape, kernel = (1, 5, 8, 9, 2, 32), (3, 1, 3)
    q, k, v, g = make(shape, 59, scale)
    o = dict(softcap=softcap, slopes=None, doc=None, prefix=None)
    value, bound = ref.scored(q, k, v, kernel, **o)["lse"]
    got = run(q, k, v, g, kernel, o)["lse"]
    ref.check("lse", got, (value, bound + 2.0 ** -21 * softcap))


@pytest.mark.parametrize("softcap", [0.0, 5.0, 30.0, 66.0, 300.0])
@pytest.mark.parametrize("kernel", [(1, 1, 1), (3, 1, 1)])
def test_a_row_of_one_key_is_its_value(softcap, kernel):
    """A window of one position, or a clip of one frame in a window along T: out is the
    value, lse the score, to fp32 rounding (2^-18 of the magnitudes, 32 products and the
    cap in turn), dv the sum's one term. dq has nothing but what delta's fp32 sum leaves of
    dp, and dk that and (1 - p) dp: its delta is p dp, with p = e^(s - lse), where s and lse
    are off by ten roundings between them, 2^-20 of themselves."""
    shape = (1, 5, 7, 10, 2, 32)
    q, k, v, g = make(shape, 61, 2.0)
    o = dict(softcap=softcap, slopes=None, prefix=None, doc=torch.arange(5, dtype=torch.int32)[None, :, None, None].expand(shape[:4]).contiguous())
    got = run(q, k, v, g, kernel, o)
    a, mag = (q.double() * k.double()).sum(-1), (q.double() * k.double()).abs().sum(-1)
    lse = softcap * torch.tanh(a / softcap) if softcap else a
    assert torch.equal(got["out"].cpu(), v)
    assert torch.equal(got["dv"].cpu(), g)
    assert bool(((got["lse"].cpu() - lse).abs() <= 2.0 ** -18 * mag).all())
    left = 2.0 ** -18 * (g.double() * v.double()).abs().sum(-1, keepdim=True)
    assert bool((got["dq"].cpu().abs() <= left * k.double().abs()).all())
    left = left * (1 + lse.abs()[..., None] / 4)
    assert bool((got["dk"].cpu().abs() <= left * q.double().abs()).all())


@pytest.mark.parametrize("softcap", [0.0, 5.0, 30.0])
@pytest.mark.parametrize("kernel", [(1, 1, 1), (1, 3, 1), (5, 1, 1)])
def test_dq_of_few_keys_is_off_by_its_rounding(kernel, softcap):
    """Over few keys dq does not take the rounding of out, which delta would bring: it is off
    by half a step and by fp32 arithmetic. With sums of 16 products 2^-20 of their magnitudes
    off, a score is by 2^-19 of its own and 2^-21 of the cap (o), p by 2 o, and da by p |dp|
    times 6 o and 2^-15 for its second bf16 part, the cap's slope and the sum of p dp."""
    T, H, W, NH, HD = shape = (7, 9, 12, 2, 16)
    q, k, v, g = make((1, *shape), 67, 2.0)
    o = make_options((1, *shape), 67, softcap, False, 2, 1)
    got = run(q, k, v, g, kernel, o)["dq"].cpu().double()
    want, _ = ref.scored(q, k, v, kernel, dout=g, **o)["dq"]
    idx = ref.window_index(T, H, W, kernel)
    aq, ak, av, ag = (x.double().abs().reshape(-1, NH, HD) for x in (q, k, v, g))
    off = 2.0 ** -19 * torch.einsum("nhd,nkhd->nkh", aq, ak[idx]).amax(1) + 2.0 ** -21 * softcap
    dp = torch.einsum("nhd,nkhd->nkh", ag, av[idx]).amax(1)
    bound = ((6 * off + 2.0 ** -15) * dp)[..., None] * ak[idx].amax(1)
    bound = ref.HALF * want.abs() + bound.reshape(want.shape)
    assert bool(((got - want).abs() <= bound).all())


def test_small_window_backward_in_a_graph():
    """Both of its passes for dQ, captured and replayed on other inputs."""
    shape, kernel = (1, 6, 9, 11, 2, 32), (1, 3, 1)
    dev = [x.cuda() for x in make(shape, 71)]
    out, lse = torch.empty_like(dev[0]), torch.empty(shape[:5], device="cuda")
    grads = [torch.empty_like(dev[0]) for _ in range(3)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        na.na3d_scored_fwd(*dev[:3], out, kernel, lse, softcap=9.0)
        na.na3d_scored_bwd(*dev[:3], out, lse, dev[3], *grads, kernel, softcap=9.0)
    for seed in (72, 73):
        new = make(shape, seed)
        for d, s in zip(dev, new):
            d.copy_(s)
        graph.replay()
        torch.cuda.synchronize()
        want = ref.scored(*new[:3], kernel, dout=new[3], softcap=9.0)
        for name, x in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *grads)):
            ref.check(name, x, want[name])
