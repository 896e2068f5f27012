"""What is measured of the score-shaped neighbourhood attention and the QKV projection with adapters.

Two operators of a batch that packs several requests into one tensor:

* the projection gives every request's tokens its own low-rank adapter beside the shared weight
  (``na3d_lora_qkv_proj``; training: ``na3d_lora_qkv_proj_bwd``);
* the attention over 3-D windows keeps the requests apart by a document mask, and takes a tanh cap on the
  scores, a bias that falls with the distance and a causal mask with a free prefix along T
  (``na3d_scored_attention``; training: ``na3d_scored_bwd``).

``run`` computes them in elementary torch operations in 32 bits, or, where ``own`` is true, through the
library's entry points.
"""
import math

import torch

own = False

# The largest attention case gathers this many key values (tokens * window * heads * head dim), the largest
# training case that many, and the largest projection multiplies M * C * N.
FWD_MOST = 65536 * 147 * 512
BWD_MOST = 24576 * 147 * 512
PROJ_MOST = 49152 * 2048 * 6144
PROJ_BWD_MOST = 65536 * 512 * 1536


def _attn(name, op, shape, kernel, softcap=0.0, slopes=False, docs=0, pad=0, prefix=-1):
    """op: "attn" or "attn_train"; docs: clips packed along T (0: no document mask); pad: padded columns at
    the end of W (document -1); prefix: leading frames that every frame sees, -1 without the causal mask."""
    case = dict(zip(("B", "T", "H", "W", "NH", "HD", "KT", "KH", "KW"), (*shape, *kernel)))
    case.update(op=op, softcap=softcap, slopes=slopes, docs=docs, pad=pad, prefix=prefix)
    return dict(case, name=name) if name else case


def _proj(name, op, M, C, NH, HD, R, requests, adapters, bias=True):
    """op: "proj" or "proj_train"; M tokens of `requests` requests, rank R, `adapters` adapters."""
    case = dict(op=op, M=M, C=C, NH=NH, HD=HD, R=R, requests=requests, adapters=adapters, bias=bias)
    return dict(case, name=name) if name else case


def listed():
    return [
        # one small latent tile: the call's own latency
        _attn("attn tiny", "attn", (1, 4, 8, 16, 2, 32), (3, 5, 5), 20.0, True, 2, 0),
        # a decoder level of one clip: capped scores with the distance bias
        _attn("attn clip 3x7x7", "attn", (1, 16, 64, 64, 8, 64), (3, 7, 7), 30.0, True),
        # whole-row windows, two clips packed along T, the last columns padded
        _attn("attn rows 3x7x33", "attn", (1, 8, 64, 33, 8, 64), (3, 7, 33), 0.0, True, 2, 3),
        # head dim 128: causal along T after two conditioning frames, packed clips, no cap
        _attn("attn hd128 causal", "attn", (1, 8, 48, 64, 16, 128), (3, 7, 7), 0.0, False, 2, 0, 2),
        # a wide window on a small odd grid
        _attn("attn 11x11x11", "attn", (1, 13, 20, 21, 8, 64), (11, 11, 11), 50.0, False, 1, 2),
        # training: forward and gradients of one clip
        _attn("attn train 3x7x7", "attn_train", (1, 16, 32, 48, 8, 64), (3, 7, 7), 30.0, True),
        # training on a padded packed batch with odd sizes
        _attn("attn train odd", "attn_train", (2, 6, 13, 21, 4, 32), (3, 5, 7), 15.0, True, 2, 4, 1),
        # eight requests of one token each, an adapter of its own for each
        _proj("proj 8 tokens", "proj", 8, 2048, 16, 128, 16, 8, 8),
        # four clips in one batch on the 512-channel decoder level
        _proj("proj clips c512", "proj", 65536, 512, 8, 64, 32, 4, 3),
        # the 2048-channel level, rank 64
        _proj("proj clips c2048", "proj", 49152, 2048, 16, 128, 64, 6, 5),
        # training of the adapters of four clips
        _proj("proj train c512", "proj_train", 65536, 512, 8, 64, 16, 4, 3, False),
        # training on many short requests of odd lengths
        _proj("proj train odd", "proj_train", 1777, 264, 3, 32, 24, 13, 5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _odd(rng, most):
    return 2 * rng.randrange((most + 1) // 2) + 1


def draw(rng):
    op = rng.choice(("attn", "attn", "attn_train", "proj", "proj", "proj_train"))
    if op.startswith("attn"):
        most = FWD_MOST if op == "attn" else BWD_MOST
        while True:
            T, H, W = _log(rng, 1, 20), _log(rng, 1, 80), _log(rng, 1, 110)
            kernel = (_odd(rng, min(T, 7)), _odd(rng, min(H, 13)), _odd(rng, min(W, 35)))
            shape = (rng.choice((1, 1, 2, 3)), T, H, W, rng.randint(1, 12), rng.choice((16, 32, 64, 64, 128)))
            size = shape[0] * T * H * W * shape[4] * shape[5] * kernel[0] * kernel[1] * kernel[2]
            if 40000 <= size <= most:
                break
        docs = rng.choice((0, 1, 2, 3))
        return _attn(None, op, shape, kernel, rng.choice((0.0, 0.0, 15.0, 30.0, 50.0)), rng.random() < 0.5,
                     docs, rng.randrange(0, max(1, W // 4)) if docs else 0, rng.choice((-1, -1, 0, 1, 3)))
    most = PROJ_MOST if op == "proj" else PROJ_BWD_MOST
    while True:
        M, C = _log(rng, 1, 65536), 8 * _log(rng, 4, 256)
        NH, HD = _log(rng, 1, 16), rng.choice((16, 32, 64, 128))
        if M * C * 3 * NH * HD <= most:
            break
    return _proj(None, op, M, C, NH, HD, 8 * _log(rng, 1, 16), _log(rng, 1, min(M, 40)), rng.randint(1, 8), rng.random() < 0.5)


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    randn = lambda *shape: torch.randn(shape, generator=gen, device="cuda")  # noqa: E731
    if case["op"].startswith("attn"):
        B, T, H, W, NH, HD = (case[n] for n in ("B", "T", "H", "W", "NH", "HD"))
        # q, k and v are the views of a fused projection's output, q scaled by HD^-0.5
        qkv = randn(B, T, H, W, 3, NH, HD)
        qkv[..., 0, :, :] *= HD ** -0.5
        s = {"op": case["op"], "kernel": (case["KT"], case["KH"], case["KW"]), "softcap": case["softcap"],
             "qkv": qkv.to(torch.bfloat16), "slopes": None, "doc": None, "prefix": None}
        if case["slopes"]:
            # 2^-1 ... 2^-4 over the heads, half of it along T
            e = torch.arange(NH, device="cuda", dtype=torch.float32) / max(1, NH - 1)
            s["slopes"] = (2.0 ** (-1 - 3 * e))[:, None] * torch.tensor([0.5, 1.0, 1.0], device="cuda")
        if case["docs"]:
            # clips of differing lengths along T, per batch entry; the padded columns belong to none
            cuts = torch.randint(0, T + 1, (B, case["docs"] - 1), generator=gen, device="cuda")
            doc = (torch.arange(T, device="cuda")[None, :, None] >= cuts[:, None, :]).sum(-1)
            doc = doc[:, :, None, None].expand(B, T, H, W).to(torch.int32).contiguous()
            if case["pad"]:
                doc[..., W - case["pad"]:] = -1
            s["doc"] = doc
        if case["prefix"] >= 0:
            s["prefix"] = torch.full((B,), case["prefix"], dtype=torch.int32, device="cuda")
        if case["op"] == "attn_train":
            s["dout"] = randn(B, T, H, W, NH, HD).to(torch.bfloat16)
        return s
    M, C, R, NH, HD = (case[n] for n in ("M", "C", "R", "NH", "HD"))
    N, n_req, n_ad = 3 * NH * HD, case["requests"], case["adapters"]
    # requests of differing lengths, none empty where there are rows enough; one in eight has no adapter
    cuts = torch.randperm(M - 1, generator=gen, device="cuda")[:n_req - 1].sort().values + 1 if n_req > 1 else \
        torch.zeros(0, dtype=torch.int64, device="cuda")
    ends = torch.tensor([M], device="cuda")
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), cuts, ends]).to(torch.int32)
    adapter = torch.randint(0, n_ad, (n_req,), generator=gen, device="cuda")
    adapter = torch.where(torch.rand(n_req, generator=gen, device="cuda") < 0.125, -1, adapter).to(torch.int32)
    s = {"op": case["op"], "NH": NH, "HD": HD, "offsets": offsets, "adapter": adapter,
         "x": randn(M, C).to(torch.bfloat16), "w": (randn(N, C) * C ** -0.5).to(torch.bfloat16),
         "bias": (0.5 * randn(N)).to(torch.bfloat16) if case["bias"] else None,
         "lora_a": (randn(n_ad, R, C) * C ** -0.5).to(torch.bfloat16),
         "lora_b": (randn(n_ad, N, R) * R ** -0.5).to(torch.bfloat16),
         "scaling": torch.linspace(0.5, 1.0, n_ad, device="cuda")}
    if case["op"] == "proj_train":
        s["dqkv"] = randn(M, N).to(torch.bfloat16)
    return s


# ------------------------------------------------------------------ the plain forms

def _window_index(T, H, W, kernel):
    """(T*H*W, KT*KH*KW) token numbers of every query's window, shifted inward at the borders."""
    axes = []
    for n, k in zip((T, H, W), kernel):
        start = (torch.arange(n, device="cuda") - k // 2).clamp(0, n - k)
        axes.append(start[:, None] + torch.arange(k, device="cuda"))
    t, h, w = axes
    idx = (t[:, None, None, :, None, None] * H + h[None, :, None, None, :, None]) * W + w[None, None, :, None, None, :]
    return idx.reshape(T * H * W, -1)


def _plain_attn(s):
    qkv, kernel = s["qkv"], s["kernel"]
    B, T, H, W, _, NH, HD = qkv.shape
    n = T * H * W
    q, k, v = (qkv[..., j, :, :].reshape(B, n, NH, HD).float() for j in range(3))
    idx = _window_index(T, H, W, kernel)
    kw = k[:, idx]                                               # (B, n, keys, NH, HD)
    sc = torch.einsum("bnkhd,bnhd->bnkh", kw, q)
    cap = None
    if s["softcap"]:
        cap = torch.tanh(sc / s["softcap"])
        sc = s["softcap"] * cap
    if s["slopes"] is not None:
        pos = torch.stack([torch.arange(n, device="cuda") // (H * W), torch.arange(n, device="cuda") // W % H,
                           torch.arange(n, device="cuda") % W], -1)
        sc = sc - (pos[idx] - pos[:, None]).abs().float() @ s["slopes"].t()
    seen = torch.ones((B, n, idx.shape[1]), dtype=torch.bool, device="cuda")
    if s["doc"] is not None:
        doc = s["doc"].reshape(B, n)
        seen = (doc[:, idx] == doc[:, :, None]) & (doc >= 0)[:, :, None]
    if s["prefix"] is not None:
        frame = torch.arange(n, device="cuda") // (H * W)
        seen = seen & ((frame[idx] <= frame[:, None])[None] | (frame[idx][None] < s["prefix"][:, None, None]))
    sc = sc.masked_fill(~seen[..., None], -math.inf)
    top = sc.amax(2, keepdim=True)
    top = torch.where(torch.isinf(top), 0.0, top)
    p = torch.exp(sc - top)
    total = p.sum(2, keepdim=True)
    lse = (top + torch.log(total)).reshape(B, T, H, W, NH)
    p = p / torch.where(total == 0, 1.0, total)
    vw = v[:, idx]
    out = torch.einsum("bnkh,bnkhd->bnhd", p, vw).to(torch.bfloat16).reshape(B, T, H, W, NH, HD)
    if s["op"] == "attn":
        return out, lse
    dout = s["dout"].reshape(B, n, NH, HD).float()
    dp = torch.einsum("bnhd,bnkhd->bnkh", dout, vw)
    ds = p * (dp - (p * dp).sum(2, keepdim=True))
    if cap is not None:
        ds = ds * (1 - cap * cap)
    dq = torch.einsum("bnkh,bnkhd->bnhd", ds, kw)
    flat = idx.reshape(-1)
    dk = torch.zeros_like(k).index_add_(1, flat, (ds[..., None] * q[:, :, None]).reshape(B, -1, NH, HD))
    dv = torch.zeros_like(v).index_add_(1, flat, (p[..., None] * dout[:, :, None]).reshape(B, -1, NH, HD))
    return out, lse, torch.stack([dq, dk, dv], 2).to(torch.bfloat16).reshape(qkv.shape)


def _plain_proj(s):
    x, w, a, b = (s[n].float() for n in ("x", "w", "lora_a", "lora_b"))
    M, (n_ad, R, C), N = x.shape[0], a.shape, w.shape[0]
    scale = torch.ones(N, device="cuda")
    scale[:N // 3] = s["HD"] ** -0.5
    # the scaling of the row's adapter in its column, 0 elsewhere
    req = torch.searchsorted(s["offsets"][1:], torch.arange(M, device="cuda", dtype=torch.int32), right=True)
    pick = (s["adapter"][req][:, None] == torch.arange(n_ad, device="cuda")) * s["scaling"]
    t = ((x @ a.reshape(n_ad * R, C).t()).reshape(M, n_ad, R) * pick[:, :, None]).reshape(M, n_ad * R)
    b_rows = b.permute(0, 2, 1).reshape(n_ad * R, N)
    if s["op"] == "proj":
        y = x @ w.t() + t @ b_rows
        if s["bias"] is not None:
            y = y + s["bias"].float()
        return (y * scale).to(torch.bfloat16)
    g = s["dqkv"].float() * scale
    u = ((g @ b_rows.t()).reshape(M, n_ad, R) * pick[:, :, None]).reshape(M, n_ad * R)
    dx = g @ w + u @ a.reshape(n_ad * R, C)
    da = (u.t() @ x).reshape(n_ad, R, C)
    db = (g.t() @ t).reshape(N, n_ad, R).permute(1, 0, 2)
    return dx.to(torch.bfloat16), da.to(torch.bfloat16), db.to(torch.bfloat16).contiguous()


def run(state):
    s = state
    if not own:
        return _plain_attn(s) if s["op"].startswith("attn") else _plain_proj(s)
    import neighborhood_attention_video_gb300 as na
    if s["op"].startswith("attn"):
        q, k, v = na.qkv_views(s["qkv"])
        shape = dict(softcap=s["softcap"], slopes=s["slopes"], doc=s["doc"], prefix=s["prefix"])
        out, lse = na.na3d_scored_attention(q, k, v, s["kernel"], return_lse=True, **shape)
        if s["op"] == "attn":
            return out, lse
        dqkv = torch.empty_like(s["qkv"])
        na.na3d_scored_bwd(q, k, v, out, lse, s["dout"], *na.qkv_views(dqkv), s["kernel"], **shape)
        return out, lse, dqkv
    adapters = (s["lora_a"], s["lora_b"], s["scaling"], s["offsets"], s["adapter"])
    if s["op"] == "proj":
        qkv = torch.empty((s["x"].shape[0], s["w"].shape[0]), dtype=torch.bfloat16, device="cuda")
        na.na3d_lora_qkv_proj(s["x"], s["w"], s["bias"], *adapters, qkv, s["NH"], s["HD"])
        return qkv
    dx, da, db = (torch.empty_like(s[n]) for n in ("x", "lora_a", "lora_b"))
    na.na3d_lora_qkv_proj_bwd(s["dqkv"], s["x"], s["w"], *adapters, dx, da, db, s["NH"], s["HD"])
    return dx, da, db


def work(case):
    if case["op"].startswith("attn"):
        n = case["B"] * case["T"] * case["H"] * case["W"]
        values = n * case["NH"] * case["HD"]
        # q k^T and p v; backward: the scores again, dp, dq, dk and dv
        flops = 4 * values * case["KT"] * case["KH"] * case["KW"]
        read_written = 8 * values + 4 * n * case["NH"] + (4 * n if case["docs"] else 0)
        if case["op"] == "attn_train":
            # the backward pass reads q, k, v, out, dout and lse again and writes the three gradients
            return {"bytes": read_written + 16 * values + 4 * n * case["NH"], "flops": flops + 10 * values * case["KT"] * case["KH"] * case["KW"]}
        return {"bytes": read_written, "flops": flops}
    M, C, R, N, n_ad = case["M"], case["C"], case["R"], 3 * case["NH"] * case["HD"], min(case["adapters"], case["requests"])
    weights = 2 * (N * C + n_ad * R * (C + N))
    if case["op"] == "proj":
        return {"bytes": weights + 2 * M * (C + N) + (2 * N if case["bias"] else 0), "flops": 2 * M * (C * N + R * (C + N))}
    # dqkv, x, the weights and adapters read; dx and the adapters' gradients written
    return {"bytes": weights + 2 * M * (2 * C + N) + 2 * case["adapters"] * R * (C + N), "flops": 2 * M * (C * N + 4 * R * (C + N))}


# ------------------------------------------------------------------ 64 bits

def _exact_attn(case, s):
    """One window slot after another, in 64 bits: slot (a, b, c) is the key at (start_t + a, start_h + b,
    start_w + c) of every query at once."""
    f64, dev = torch.float64, "cuda"
    B, T, H, W, NH, HD = (case[n] for n in ("B", "T", "H", "W", "NH", "HD"))
    q, k, v = (s["qkv"][:, :, :, :, j].to(f64) for j in range(3))
    pos = [torch.arange(n, device=dev) for n in (T, H, W)]
    first = [torch.clamp(torch.clamp(p - K // 2, min=0), max=n - K) for p, K, n in zip(pos, s["kernel"], (T, H, W))]
    slots = [(a, b, c) for a in range(case["KT"]) for b in range(case["KH"]) for c in range(case["KW"])]

    def at(x, a, b, c):
        return x.index_select(1, first[0] + a).index_select(2, first[1] + b).index_select(3, first[2] + c)

    scores = torch.empty((len(slots), B, T, H, W, NH), dtype=f64, device=dev)
    slope = []
    for i, (a, b, c) in enumerate(slots):
        sc = (q * at(k, a, b, c)).sum(-1)
        if s["softcap"]:
            th = torch.tanh(sc / s["softcap"])
            slope.append(1 - th ** 2 if case["op"] == "attn_train" else None)
            sc = s["softcap"] * th
        if s["slopes"] is not None:
            sl = s["slopes"].to(f64)
            far = [(f + o - p).abs().to(f64) for f, o, p in zip(first, (a, b, c), pos)]
            sc = sc - (far[0][:, None, None, None] * sl[:, 0] + far[1][None, :, None, None] * sl[:, 1] +
                       far[2][None, None, :, None] * sl[:, 2])
        if s["doc"] is not None:
            theirs = at(s["doc"], a, b, c)
            sc[((theirs != s["doc"]) | (theirs < 0))] = -math.inf
        if s["prefix"] is not None:
            late = (first[0] + a)[None] > pos[0][None]
            late = late & ((first[0] + a)[None] >= s["prefix"][:, None])
            sc[late[:, :, None, None, None].expand_as(sc)] = -math.inf
        scores[i] = sc
    lse = torch.logsumexp(scores, 0)
    weight = lambda i: torch.where(torch.isinf(lse), 0.0, torch.exp(scores[i] - lse))  # noqa: E731
    out = torch.zeros_like(q)
    for i, at_ in enumerate(slots):
        out += weight(i)[..., None] * at(v, *at_)
    if case["op"] == "attn":
        return out, lse
    dout = s["dout"].to(f64)
    inner = (dout * out).sum(-1)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for i, (a, b, c) in enumerate(slots):
        p = weight(i)
        ds = p * ((dout * at(v, a, b, c)).sum(-1) - inner)
        if slope:
            ds = ds * slope[i]
        dq += ds[..., None] * at(k, a, b, c)
        token = (((first[0] + a) * H)[:, None, None] + (first[1] + b)[None, :, None]) * W + (first[2] + c)
        dk.view(B, T * H * W, NH, HD).index_add_(1, token.reshape(-1), (ds[..., None] * q).view(B, -1, NH, HD))
        dv.view(B, T * H * W, NH, HD).index_add_(1, token.reshape(-1), (p[..., None] * dout).view(B, -1, NH, HD))
    return out, lse, torch.stack([dq, dk, dv], 4)


def _exact_proj(case, s):
    """One request after another, in 64 bits."""
    f64 = torch.float64
    x, w = s["x"].to(f64), s["w"].to(f64)
    M, C, N, n_q = case["M"], case["C"], w.shape[0], case["NH"] * case["HD"]
    ends, ids, by = s["offsets"].tolist(), s["adapter"].tolist(), s["scaling"].tolist()
    if case["op"] == "proj":
        y = x @ w.t()
        for r, i in enumerate(ids):
            if i >= 0:
                rows = slice(ends[r], ends[r + 1])
                y[rows] += by[i] * ((x[rows] @ s["lora_a"][i].to(f64).t()) @ s["lora_b"][i].to(f64).t())
        if s["bias"] is not None:
            y += s["bias"].to(f64)
        y[:, :n_q] /= math.sqrt(case["HD"])
        return y
    g = s["dqkv"].to(f64)
    g[:, :n_q] /= math.sqrt(case["HD"])
    dx = g @ w
    da, db = (torch.zeros(s[n].shape, dtype=f64, device="cuda") for n in ("lora_a", "lora_b"))
    for r, i in enumerate(ids):
        if i >= 0:
            rows = slice(ends[r], ends[r + 1])
            a, b = s["lora_a"][i].to(f64), s["lora_b"][i].to(f64)
            back = by[i] * (g[rows] @ b)
            dx[rows] += back @ a
            da[i] += back.t() @ x[rows]
            db[i] += by[i] * (g[rows].t() @ (x[rows] @ a.t()))
    return dx, da, db


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_attn(case, s) if case["op"].startswith("attn") else _exact_proj(case, s)
