"""The projection with adapters on the GPU against the 64-bit reference, forward
and backward, and feeding the score-shaped attention."""
import pytest
import torch

import neighborhood_attention_video_gb300 as na
import packed_reference as ref

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def make(M, C, NH, HD, R, n_ad, seed, bias=True):
    gen = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    N = 3 * NH * HD
    t = dict(x=rand(M, C), w=rand(N, C) * C ** -0.5, bias=rand(N) if bias else None,
             lora_a=rand(n_ad, R, C) * C ** -0.5, lora_b=rand(n_ad, N, R) * R ** -0.5)
    t = {n: v.to(BF16) if v is not None else None for n, v in t.items()}
    t["scaling"] = torch.rand(n_ad, generator=gen) + 0.5
    return t, rand(M, N).to(BF16)


def ints(*v):
    return torch.tensor(v, dtype=torch.int32)


def run(t, dqkv, offsets, adapter, NH, HD, want_dx=True, **kw):
    d = {n: v.cuda() if v is not None else None for n, v in t.items()}
    M, N = dqkv.shape
    off, ad = offsets.cuda(), adapter.cuda()
    adapters = (d["lora_a"], d["lora_b"], d["scaling"], off, ad)
    nan = lambda x: torch.full_like(x, float("nan"))  # noqa: E731
    qkv = nan(dqkv.cuda())
    grad = dqkv.cuda()
    torch.cuda.synchronize()
    na.na3d_lora_qkv_proj(d["x"], d["w"], d["bias"], *adapters, qkv, NH, HD, **kw)
    dx, da, db = nan(d["x"]) if want_dx else None, nan(d["lora_a"]), nan(d["lora_b"])
    torch.cuda.synchronize()
    na.na3d_lora_qkv_proj_bwd(grad, d["x"], d["w"], *adapters, dx, da, db, NH, HD, **kw)
    torch.cuda.synchronize()
    assert na.na3d_device_status() == 0
    return dict(qkv=qkv, da=da, db=db, **({"dx": dx} if want_dx else {}))


CASES = [
    # M, C, NH, HD, R, n_ad, offsets, adapters
    (1, 64, 2, 32, 8, 1, (0, 1), (0,)),
    (1, 8, 1, 16, 8, 2, (0, 1), (-1,)),
    (5, 264, 3, 32, 16, 5, (0, 1, 2, 3, 4, 5), (4, 0, 4, -1, 2)),      # single tokens, an adapter twice
    (8, 2048, 4, 128, 16, 8, tuple(range(9)), tuple(range(8))),
    (32, 1024, 2, 64, 8, 3, (0, 31, 32), (2, 0)),
    (33, 512, 8, 64, 64, 3, (0, 7, 7, 20, 33), (1, 2, 1, 0)),          # an empty request
    (64, 136, 5, 16, 40, 2, (3, 10, 60), (1, 0)),                      # rows outside every request
    (100, 64, 2, 32, 8, 2, (0, 100), (7,)),                            # an id past the adapters: none
    (128, 512, 8, 64, 32, 2, (0, 64, 128), (0, 1)),
    (129, 72, 2, 64, 128, 2, (0, 128, 129), (0, 1)),
    (300, 96, 3, 16, 24, 4, (0, 1, 2, 130, 131, 257, 299), (3, 2, 1, 0, 3, 3)),
    (777, 256, 4, 128, 16, 2, (0, 300, 777), (1, 1)),                  # one adapter throughout
    (1000, 1032, 1, 64, 72, 3, (10, 20, 500, 990), (0, -1, 2)),
    (2500, 520, 3, 32, 32, 4, (0, 1000, 1001, 2499, 2500), (2, 3, 0, 2)),
    # enough rows for tiles of 256 by pairs of blocks
    (20045, 72, 3, 32, 24, 3, (5, 100, 300, 384, 9001, 20000), (0, 2, 1, 0, 2)),
    (20045, 264, 2, 16, 128, 2, (0, 10000, 20045), (1, 0)),
    (19456, 328, 1, 128, 64, 1, (0, 19456), (0,)),
    # and more of them: six tiles for each pair
    (58477, 264, 3, 32, 24, 3, (5, 100, 300, 384, 9001, 58400), (0, 2, 1, 0, 2)),
    (30001, 776, 5, 64, 128, 2, (0, 10000, 30001), (1, 0)),
    (25600, 136, 3, 128, 64, 1, (0, 25600), (0,)),
]


@pytest.mark.parametrize("M,C,NH,HD,R,n_ad,offsets,adapter", CASES, ids=lambda v: str(v).replace(" ", ""))
def test_matches_the_reference(M, C, NH, HD, R, n_ad, offsets, adapter):
    t, g = make(M, C, NH, HD, R, n_ad, M + C + R, bias=M % 2 == 0)
    off, ad = ints(*offsets), ints(*adapter)
    want = ref.lora(**t, offsets=off, adapter=ad, HD=HD, dqkv=g)
    got = run(t, g, off, ad, NH, HD)
    for name in want:
        ref.check(name, got[name], want[name])


def test_random_problems():
    gen = torch.Generator().manual_seed(6)
    upto = lambda n: 1 + int(torch.randint(0, n, (1,), generator=gen))  # noqa: E731
    for i in range(30):
        M = upto((8, 40, 150, 700)[i % 4])
        C, NH, HD, R = 8 * upto(40), upto(6), (16, 32, 64, 128)[upto(4) - 1], 8 * upto(16)
        n_ad, n_req = upto(5), upto(9)
        off = torch.randint(0, M + 1, (n_req + 1,), generator=gen).sort().values.to(torch.int32)
        ad = torch.randint(-1, n_ad + 1, (n_req,), generator=gen).to(torch.int32)
        t, g = make(M, C, NH, HD, R, n_ad, i, bias=i % 2 == 0)
        want = ref.lora(**t, offsets=off, adapter=ad, HD=HD, dqkv=g)
        got = run(t, g, off, ad, NH, HD, want_dx=i % 3 != 0)
        for name in got:
            ref.check(f"problem {i} M={M} C={C} NH={NH} HD={HD} R={R} {name}", got[name], want[name])


def test_without_adapters_it_is_the_base_projection():
    """Where no request has an adapter, the values of na3d_qkv_proj."""
    M, C, NH, HD = 700, 256, 4, 64
    t, g = make(M, C, NH, HD, 16, 2, 1)
    got = run(t, g, ints(0, 300, 700), ints(-1, -1), NH, HD)
    base = torch.empty_like(got["qkv"])
    na.na3d_qkv_proj(t["x"].cuda(), t["w"].cuda(), t["bias"].cuda(), base, NH, HD)
    want = ref.lora(**t, offsets=ints(0, 300, 700), adapter=ints(-1, -1), HD=HD)["qkv"]
    ref.check("qkv", got["qkv"], want)
    ref.check("base", base, want)
    assert bool((got["da"] == 0).all()) and bool((got["db"] == 0).all())


@pytest.mark.parametrize("M", [6, 150, 20000, 58600])
def test_requests_do_not_reach_one_another(M):
    """A request's rows are what they are by themselves whatever the other
    requests, their adapters included, hold."""
    C, NH, HD = 264 if M > 50000 else 128, 2, 64   # pairs of blocks in both directions
    t, g = make(M, C, NH, HD, 16, 2, 2)
    cuts = (0, 2, 4, 6) if M == 6 else (0, 50, 100, M)
    off, ad = ints(*cuts), ints(0, 1, 0)
    clean = run(t, g, off, ad, NH, HD)
    want = ref.lora(**t, offsets=off, adapter=ad, HD=HD, dqkv=g)
    t["x"][cuts[1]:cuts[2]] = float("nan")
    t["lora_a"][1] = float("nan")
    t["lora_b"][1] = float("inf")
    got = run(t, g, off, ad, NH, HD)
    for rows in (slice(0, cuts[1]), slice(cuts[2], M)):
        for name in ("qkv", "dx"):
            value, bound = want[name]
            ref.check(name, got[name][rows], (value[rows], bound[rows]))
    for name in ("da", "db"):
        assert torch.equal(got[name][0], clean[name][0]), name


@pytest.mark.parametrize("M,n_req", [(3000, 1500), (20, 2000), (19500, 40), (58600, 1100)])
def test_many_requests(M, n_req):
    """More requests than a block keeps at hand, most of them empty or of one row."""
    gen = torch.Generator().manual_seed(M)
    C, NH, HD, R, n_ad = 264 if M > 50000 else 64, 2, 64, 16, 7
    off = torch.randint(0, M + 1, (n_req + 1,), generator=gen).sort().values.to(torch.int32)
    ad = torch.randint(-1, n_ad, (n_req,), generator=gen).to(torch.int32)
    t, g = make(M, C, NH, HD, R, n_ad, 9)
    want = ref.lora(**t, offsets=off, adapter=ad, HD=HD, dqkv=g)
    got = run(t, g, off, ad, NH, HD)
    for name in want:
        ref.check(name, got[name], want[name])


def test_two_streams_at_once():
    """Calls on two streams, each with a workspace of its own."""
    C, NH, HD = 128, 2, 64
    off, ad = ints(0, 100, 900), ints(1, 0)
    data = [make(900, C, NH, HD, 16, 2, s) for s in (1, 2)]
    want = [ref.lora(**t, offsets=off, adapter=ad, HD=HD, dqkv=g) for t, g in data]
    streams = [torch.cuda.Stream() for _ in data]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    results = [None, None]
    for _ in range(5):
        for i, (t, g) in enumerate(data):
            with torch.cuda.stream(streams[i]):
                d = {n: v.cuda() for n, v in t.items()}
                adapters = (d["lora_a"], d["lora_b"], d["scaling"], off.cuda(), ad.cuda())
                qkv = torch.empty((900, 3 * NH * HD), dtype=BF16, device="cuda")
                na.na3d_lora_qkv_proj(d["x"], d["w"], d["bias"], *adapters, qkv, NH, HD)
                dx, da, db = (torch.empty_like(d[n]) for n in ("x", "lora_a", "lora_b"))
                na.na3d_lora_qkv_proj_bwd(g.cuda(), d["x"], d["w"], *adapters, dx, da, db, NH, HD)
                results[i] = dict(qkv=qkv, dx=dx, da=da, db=db)
    torch.cuda.synchronize()
    for w, r in zip(want, results):
        for name in w:
            ref.check(name, r[name], w[name])


def test_stream_argument():
    """stream= of another stream than the current one; the binding's own workspace."""
    C, NH, HD = 64, 1, 64
    t, g = make(200, C, NH, HD, 16, 2, 3)
    off, ad = ints(0, 90, 200), ints(1, 0)
    want = ref.lora(**t, offsets=off, adapter=ad, HD=HD, dqkv=g)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = run(t, g, off, ad, NH, HD, stream=side)
    for name in want:
        ref.check(name, got[name], want[name])


def test_offsets_out_of_order_touch_nothing_else():
    """Offsets that decrease or leave the rows: every output is written, inside its tensor."""
    M, C, NH, HD = 200, 64, 2, 32
    t, g = make(M, C, NH, HD, 16, 2, 3)
    for off in (ints(0, 150, 50, 400), ints(-7, 20, 20, 10), ints(300, 200, 100, 0), ints(250, 260, 270, 280)):
        got = run(t, g, off, ints(0, 1, 0), NH, HD)
        assert all(bool(torch.isfinite(x).all()) for x in got.values())


def test_same_inputs_same_bits():
    t, g = make(1500, 264, 3, 64, 32, 3, 4)
    off, ad = ints(0, 100, 700, 1500), ints(2, 0, 2)
    first = run(t, g, off, ad, 3, 64)
    for _ in range(5):
        got = run(t, g, off, ad, 3, 64)
        assert all(torch.equal(got[n], first[n]) for n in first)


@pytest.mark.parametrize("M", [6, 300])
def test_graph_with_other_requests(M):
    """A captured forward and backward pass replayed with other requests and inputs."""
    C, NH, HD, R, n_ad = 192, 2, 64, 16, 3
    N = 3 * NH * HD
    t, g = make(M, C, NH, HD, R, n_ad, 5)
    d = {n: v.cuda() for n, v in t.items()}
    gd, off, ad = g.cuda(), ints(0, 2, 4, M).cuda(), ints(0, 1, 2).cuda()
    qkv = torch.empty((M, N), dtype=BF16, device="cuda")
    dx, da, db = (torch.empty_like(d[n]) for n in ("x", "lora_a", "lora_b"))
    works = [torch.empty(na.na3d_lora_workspace(M, C, NH, HD, R, 3, n_ad, b), dtype=torch.uint8, device="cuda")
             for b in (False, True)]
    adapters = (d["lora_a"], d["lora_b"], d["scaling"], off, ad)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        na.na3d_lora_qkv_proj(d["x"], d["w"], d["bias"], *adapters, qkv, NH, HD, work=works[0])
        na.na3d_lora_qkv_proj_bwd(gd, d["x"], d["w"], *adapters, dx, da, db, NH, HD, work=works[1])
    for seed, o, a in ((5, (0, 2, 4, M), (0, 1, 2)), (6, (1, 1, M - 1, M), (2, 0, -1))):
        t, g = make(M, C, NH, HD, R, n_ad, seed)
        for n in t:
            d[n].copy_(t[n])
        gd.copy_(g)
        off.copy_(ints(*o))
        ad.copy_(ints(*a))
        graph.replay()
        torch.cuda.synchronize()
        want = ref.lora(**t, offsets=ints(*o), adapter=ints(*a), HD=HD, dqkv=g)
        for name, x in (("qkv", qkv), ("dx", dx), ("da", da), ("db", db)):
            ref.check(name, x, want[name])


def test_output_past_32_bits():
    """More than 2^31 output elements: sampled rows at both ends."""
    M, C, NH, HD, R = 1 << 20, 64, 11, 64, 16
    N = 3 * NH * HD
    assert M * N > 2 ** 31
    t, _ = make(8, C, NH, HD, R, 2, 7)
    d = {n: v.cuda() for n, v in t.items()}
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((M, C), generator=gen, device="cuda").to(BF16)
    qkv = torch.empty((M, N), dtype=BF16, device="cuda")
    off, ad = ints(0, 1000, M - 77, M), ints(1, 0, 1)
    adapters = (d["lora_a"], d["lora_b"], d["scaling"], off.cuda(), ad.cuda())
    na.na3d_lora_qkv_proj(x, d["w"], d["bias"], *adapters, qkv, NH, HD)
    dx, da, db = torch.empty_like(x), torch.empty_like(d["lora_a"]), torch.empty_like(d["lora_b"])
    na.na3d_lora_qkv_proj_bwd(qkv, x, d["w"], *adapters, dx, da, db, NH, HD)
    assert na.na3d_device_status() == 0
    t.pop("x")
    for rows, o, a in ((slice(0, 200), (0, 200), (1,)), (slice(M - 200, M), (0, 123, 200), (0, 1))):
        want = ref.lora(x[rows].cpu(), **t, offsets=ints(*o), adapter=ints(*a), HD=HD, dqkv=qkv[rows].cpu())
        ref.check("qkv", qkv[rows], want["qkv"])
        ref.check("dx", dx[rows], want["dx"])


def test_packed_batch_trains_through_both():
    """The set as it is used: two requests with their own adapters are projected,
    attend within their own frames, and their gradients come back through the
    fused gradient tensor to x and the adapters."""
    B, T, H, W, NH, HD, C, R = 1, 6, 6, 10, 2, 64, 96, 16
    kernel, M = (3, 5, 5), 6 * 6 * 10
    t, _ = make(M, C, NH, HD, R, 2, 11)
    d = {n: v.cuda() for n, v in t.items()}
    off, ad = ints(0, 2 * H * W, M), ints(1, 0)
    doc = torch.zeros((B, T, H, W), dtype=torch.int32)
    doc[:, 2:] = 1
    gen = torch.Generator().manual_seed(1)
    dout = torch.randn((B, T, H, W, NH, HD), generator=gen).to(BF16)
    adapters = (d["lora_a"], d["lora_b"], d["scaling"], off.cuda(), ad.cuda())
    qkv = torch.empty((B, T, H, W, 3, NH, HD), dtype=BF16, device="cuda")
    na.na3d_lora_qkv_proj(d["x"], d["w"], d["bias"], *adapters, qkv, NH, HD)
    views = na.qkv_views(qkv)
    out, lse = na.na3d_scored_attention(*views, kernel, softcap=20.0, doc=doc.cuda(), return_lse=True)
    dqkv = torch.empty_like(qkv)
    na.na3d_scored_bwd(*views, out, lse, dout.cuda(), *na.qkv_views(dqkv), kernel, softcap=20.0, doc=doc.cuda())
    dx, da, db = (torch.empty_like(d[n]) for n in ("x", "lora_a", "lora_b"))
    na.na3d_lora_qkv_proj_bwd(dqkv, d["x"], d["w"], *adapters, dx, da, db, NH, HD)
    torch.cuda.synchronize()
    proj = ref.lora(**t, offsets=off, adapter=ad, HD=HD, dqkv=dqkv.cpu().reshape(M, -1))
    ref.check("qkv", qkv, proj["qkv"])
    att = ref.scored(*na.qkv_views(qkv.cpu()), kernel, softcap=20.0, doc=doc, dout=dout)
    for name, x in (("out", out), ("lse", lse), *zip(("dq", "dk", "dv"), na.qkv_views(dqkv))):
        ref.check(name, x, att[name])
    for name, x in (("dx", dx), ("da", da), ("db", db)):
        ref.check(name, x, proj[name])


def test_workspaces_of_calls_that_run_at_once():
    """Calls without a ``work`` tensor, of growing and shrinking sizes: from two
    threads on one stream and on streams of their own, and beside replays of a
    graph that captured the same call. Each gives the bits it gives by itself."""
    import threading
    sizes = [(40, 1), (3000, 2), (9, 3), (6000, 4)]
    data = []
    for M, seed in sizes:
        t, g = make(M, 256, 2, 64, 16, 2, seed)
        d = {n: v.cuda() for n, v in t.items()}
        off, ad = ints(0, M // 2, M).cuda(), ints(1, 0).cuda()
        data.append((d, g.cuda(), (d["lora_a"], d["lora_b"], d["scaling"], off, ad)))

    def call(i):
        d, g, adapters = data[i]
        qkv, dx, da, db = (torch.empty_like(x) for x in (g, d["x"], d["lora_a"], d["lora_b"]))
        na.na3d_lora_qkv_proj(d["x"], d["w"], d["bias"], *adapters, qkv, 2, 64)
        na.na3d_lora_qkv_proj_bwd(g, d["x"], d["w"], *adapters, dx, da, db, 2, 64)
        return qkv, dx, da, db

    want = [[x.clone() for x in call(i)] for i in range(4)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = call(3)
    graph.replay()
    torch.cuda.synchronize()
    wrong = []

    def work(own_stream):
        stream = torch.cuda.Stream() if own_stream else torch.cuda.default_stream()
        with torch.cuda.stream(stream):
            got = [(i, call(i)) for _ in range(6) for i in (1, 0, 3, 2)]
        stream.synchronize()
        wrong.extend(i for i, r in got for x, y in zip(r, want[i]) if not torch.equal(x, y))

    threads = [threading.Thread(target=work, args=(o,)) for o in (False, True, True)]
    for th in threads:
        th.start()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(20):
            graph.replay()
    got = [(i, call(i)) for i in (3, 1, 2, 0)]
    for th in threads:
        th.join()
    torch.cuda.synchronize()
    assert not wrong
    for i, r in got + [(3, captured)]:
        for x, y in zip(r, want[i]):
            assert torch.equal(x, y), i
    assert na.na3d_device_status() == 0


@pytest.mark.parametrize("backward", [False, True], ids=["forward by blocks", "backward by pairs"])
def test_values_by_themselves_outlast_no_wait(backward):
    """In a tile that another request's infinite adapter reaches, values are computed one by
    one, over a contraction this long for more than the two seconds that a wait of the
    tile's other roles allows: the tiles that follow get their results all the same."""
    M, HD, R = 456 * 128, 64, 16                    # three tiles for each block, six for each pair
    C, NH = (264, 800) if backward else (200000, 1)
    N = 3 * NH * HD
    t, g = make(128, C, NH, HD, R, 2, 43, bias=False)
    if backward:
        t["w"] = (t["w"].float() * (C / N) ** 0.5).to(BF16)
    tall = lambda x: torch.cat([x.cuda(), torch.zeros((M - 128, x.shape[1]), dtype=BF16, device="cuda")])  # noqa: E731
    d = {n: v.cuda() for n, v in t.items() if v is not None}
    adapters = (d["lora_a"], d["lora_b"], d["scaling"], ints(0, 64, 128, M).cuda(), ints(0, 1, -1).cuda())
    d["lora_a" if backward else "lora_b"][1] = float("inf")
    x = tall(t["x"])
    if backward:
        got = torch.full_like(x, 7.0)
        da, db = torch.empty_like(d["lora_a"]), torch.empty_like(d["lora_b"])
        na.na3d_lora_qkv_proj_bwd(tall(g), x, d["w"], *adapters, got, da, db, NH, HD)
    else:
        got = torch.full((M, N), 7.0, dtype=BF16, device="cuda")
        na.na3d_lora_qkv_proj(x, d["w"], None, *adapters, got, NH, HD)
    assert na.na3d_device_status() == 0
    assert bool((got[128:] == 0).all())
    t["x"] = t["x"][:64]
    want = ref.lora(**t, offsets=ints(0, 64), adapter=ints(0), HD=HD, dqkv=g[:64] if backward else None)
    ref.check("values", got[:64], want["dx" if backward else "qkv"])
    assert not bool(torch.isfinite(got[64:128]).any())


@pytest.mark.parametrize("M", [150, 58600])
def test_a_bad_row_is_alone(M):
    """One row of a tile with two requests is not finite: its lanes of the epilogue compute
    theirs by themselves, all other rows are what they are without it."""
    C, NH, HD = 264 if M > 50000 else 128, 3, 64   # pairs of blocks in both directions
    t, g = make(M, C, NH, HD, 16, 2, 12)
    off, ad = ints(0, 70, M), ints(0, 1)
    clean = run(t, g, off, ad, NH, HD)
    row = 40
    t["x"][row, 5] = float("nan")
    g[row, 7] = float("inf")
    got = run(t, g, off, ad, NH, HD)
    others = torch.arange(M) != row
    for name in ("qkv", "dx"):
        assert torch.equal(got[name].cpu()[others], clean[name].cpu()[others]), name
        assert not bool(torch.isfinite(got[name][row]).any()), name
    for name in ("da", "db"):
        assert torch.equal(got[name][1], clean[name][1]), name
