"""What is measured of the norm and rotation of queries and keys, and of the attention to an encoder's states.

Two operators of a block of a video model, beside the projection and the windowed attention:

* the RMS norm of each head of q and k and the rotation by the position along T, H and W, in one pass over the
  views of a fused projection (``na3d_norm_rope``; training: ``na3d_norm_rope_bwd``);
* the attention of the grid's tokens to states of another length, a prompt's or earlier frames', which packed
  clips keep apart by documents (``na3d_cross_attention``; training: ``na3d_cross_bwd``).

``run`` computes them in elementary torch operations in 32 bits, or, where ``own`` is true, through the
library's entry points.
"""
import math

import torch

own = False

# The largest listed case of each kind: values of q and k, or tokens * heads * head dim * keys.
ROPE_MOST = 393216 * 4096
ROPE_TRAIN_MOST = 49152 * 4096
CROSS_MOST = 24576 * 2048 * 6144
CROSS_TRAIN_MOST = 24576 * 2048 * 512
EPS, THETA = 1e-6, 10000.0


def _rope(name, op, shape, dims, NKV=0, interleaved=True, norm=True):
    """op: "rope" or "rope_train"; dims: values of a head that turn with t, h and w; NKV: heads of k."""
    case = dict(zip(("B", "T", "H", "W", "NH", "HD", "RT", "RH", "RW"), (*shape, *dims)))
    case.update(op=op, NKV=NKV or shape[4], interleaved=interleaved, norm=norm)
    return dict(case, name=name) if name else case


def _cross(name, op, shape, S, NKV=0, docs=0, pad=False):
    """op: "cross" or "cross_train"; docs: clips packed along T, each with states of its own (0: one for all);
    pad: the states of each clip end before its share of S does."""
    case = dict(zip(("B", "T", "H", "W", "NH", "HD"), shape))
    case.update(op=op, S=S, NKV=NKV or shape[4], docs=docs, pad=pad)
    return dict(case, name=name) if name else case


def listed():
    return [
        # a step of eight requests with one token each: the call's own latency
        _rope("rope 8 tokens", "rope", (8, 1, 1, 1, 16, 128), (44, 42, 42)),
        # one clip of the 512-channel decoder level, halves of a head as pairs
        _rope("rope clip hd64", "rope", (1, 16, 64, 64, 8, 64), (16, 24, 24), interleaved=False),
        # the two clips of the headline shape
        _rope("rope clips hd128", "rope", (2, 16, 96, 128, 16, 128), (44, 42, 42)),
        # training on one clip: forward and gradients
        _rope("rope train", "rope_train", (1, 16, 48, 64, 16, 128), (44, 42, 42)),
        # training on odd sizes, shared heads of k, the last values of a head left as they are
        _rope("rope train odd", "rope_train", (2, 6, 13, 21, 6, 32), (8, 12, 8), NKV=3),
        # eight requests with one token each and a padded prompt each
        _cross("cross 8 tokens", "cross", (8, 1, 1, 1, 16, 128), 512, pad=True),
        # one token over a long memory, four heads of q to one of k and v
        _cross("cross long memory", "cross", (1, 1, 1, 1, 16, 128), 65536, NKV=4),
        # one clip over a prompt of 512 states
        _cross("cross clip hd128", "cross", (1, 16, 48, 64, 16, 128), 512),
        # four packed clips, each with its own padded prompt
        _cross("cross packed hd64", "cross", (1, 16, 64, 64, 8, 64), 1024, docs=4, pad=True),
        # the tokens of a clip over the states of two earlier frames
        _cross("cross frames hd128", "cross", (1, 8, 48, 64, 16, 128), 6144),
        # training on one clip
        _cross("cross train", "cross_train", (1, 8, 48, 64, 16, 128), 512),
        # training on two packed clips of odd sizes, a short prompt, three heads of q to one of k and v
        _cross("cross train odd", "cross_train", (2, 6, 13, 21, 6, 32), 77, NKV=2, docs=2, pad=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rope", "rope_train", "cross", "cross", "cross_train"))
    most = {"rope": ROPE_MOST, "rope_train": ROPE_TRAIN_MOST, "cross": CROSS_MOST, "cross_train": CROSS_TRAIN_MOST}[op]
    while True:
        NKV, HD = _log(rng, 1, 16), rng.choice((16, 32, 64, 64, 128, 128))
        NH = NKV * rng.choice((1, 1, 1, 2, 3, 4, 8))
        shape = (rng.choice((1, 1, 2, 3, 8)), _log(rng, 1, 20), _log(rng, 1, 96), _log(rng, 1, 128), NH, HD)
        values = shape[0] * shape[1] * shape[2] * shape[3] * HD
        if NH > 32:
            continue
        if op.startswith("rope"):
            if values * (NH + NKV) <= most:
                break
        else:
            S = _log(rng, 1, 65536)
            # the plain form holds every score in 32 bits
            if values * NH * S <= most and values // HD * NH * S <= 1 << 32:
                break
    if op.startswith("cross"):
        return _cross(None, op, shape, S, NKV, rng.choice((0, 0, 1, 2, 3)), rng.random() < 0.5)
    interleaved = rng.random() < 0.5
    if interleaved:
        h = 2 * rng.randrange(0, HD // 6 + 1)
        w = 2 * rng.randrange(0, HD // 6 + 1)
        dims = (HD - h - w - 2 * rng.randrange(0, 3), h, w)
    else:   # halves of all of the head, or of its first half
        total = HD // rng.choice((1, 1, 2)) if HD > 16 else HD
        h = 2 * rng.randrange(0, total // 6 + 1)
        w = 2 * rng.randrange(0, total // 6 + 1)
        dims = (total - h - w, h, w)
    return _rope(None, op, shape, dims, NKV, interleaved, rng.random() < 0.8)


# ------------------------------------------------------------------ inputs

def _positions(case):
    return [torch.arange(case[n], device="cuda") for n in "THW"]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    randn = lambda *shape: torch.randn(shape, generator=gen, device="cuda")  # noqa: E731
    bf16 = torch.bfloat16
    B, T, H, W, NH, HD, NKV = (case[n] for n in ("B", "T", "H", "W", "NH", "HD", "NKV"))
    s = {"op": case["op"]}
    if case["op"].startswith("rope"):
        # the output of a fused projection, a token's heads of q, k and v in a row, q scaled by HD^-0.5
        qkv = randn(B, T, H, W, NH + 2 * NKV, HD).to(bf16)
        qkv[..., :NH, :] *= HD ** -0.5
        s.update(qkv=qkv, NH=NH, NKV=NKV, norm=case["norm"], interleaved=case["interleaved"])
        s["q_scale"] = HD ** -0.5 if case["norm"] else 1.0
        s["dims"] = tuple(case[n] for n in ("RT", "RH", "RW"))
        # cos and sin of every position and frequency of an axis, laid out once for the grid
        rows = []
        for pos, R in zip(_positions(case), s["dims"]):
            if R:
                freq = THETA ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / R)
                angle = (pos[:, None] * freq).reshape(-1)
                rows.append(torch.stack([angle.cos(), angle.sin()], -1))
        s["table"] = torch.cat(rows).float() if rows else None
        if case["norm"]:
            s["q_weight"], s["k_weight"] = ((1 + 0.2 * randn(HD)).to(bf16) for _ in range(2))
        else:
            s["q_weight"] = s["k_weight"] = None
        if case["op"] == "rope_train":
            s["dq_out"], s["dk_out"] = (randn(B, T, H, W, n, HD).to(bf16) for n in (NH, NKV))
        return s
    S, docs = case["S"], case["docs"]
    s["q"] = (randn(B, T, H, W, NH, HD) * HD ** -0.5).to(bf16)
    s["kv"] = randn(B, S, 2, NKV, HD).to(bf16)       # one projection of the states
    s["doc"] = s["kv_doc"] = None
    if docs:
        # clips of differing lengths along T
        cuts = torch.randint(0, T + 1, (B, docs - 1), generator=gen, device="cuda")
        doc = (torch.arange(T, device="cuda")[None, :] >= cuts[:, :, None]).sum(1)
        s["doc"] = doc[:, :, None, None].expand(B, T, H, W).to(torch.int32).contiguous()
    if docs or case["pad"]:
        share = -(-S // max(1, docs))
        at = torch.arange(S, device="cuda")
        kv_doc = (at // share).expand(B, S)
        if case["pad"]:
            length = torch.randint(1, share + 1, (B, max(1, docs)), generator=gen, device="cuda")
            kv_doc = torch.where(at % share < length.gather(1, kv_doc), kv_doc, -1)
        s["kv_doc"] = kv_doc.to(torch.int32).contiguous()
    if case["op"] == "cross_train":
        s["dout"] = randn(B, T, H, W, NH, HD).to(bf16)
    return s


# ------------------------------------------------------------------ the plain forms

def _angles(s):
    """cos and sin (T*H*W, 1, pairs) of each token's pairs, the axes one behind another."""
    _, T, H, W = s["qkv"].shape[:4]
    parts = []
    for axis, (n, R) in enumerate(zip((T, H, W), s["dims"])):
        freq = THETA ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / max(R, 1))
        angle = torch.arange(n, device="cuda")[:, None] * freq
        view = [1, 1, 1, R // 2]
        view[axis] = n
        parts.append(angle.view(view).expand(T, H, W, R // 2))
    angle = torch.cat(parts, -1).reshape(T * H * W, 1, -1)
    return angle.cos().float(), angle.sin().float()


def _turn(x, cos, sin, interleaved):
    """x (B, T*H*W, heads, HD) with its pairs turned."""
    P = cos.shape[-1]
    if interleaved:
        a, b = x[..., 0:2 * P:2], x[..., 1:2 * P:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :P], x[..., P:2 * P]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., 2 * P:]], -1)


def _plain_rope(s):
    qkv, NH, NKV = s["qkv"], s["NH"], s["NKV"]
    B, T, H, W, _, HD = qkv.shape
    cos, sin = _angles(s)
    outs, grads, weights = [], [], []
    for name, part, eps, scale in (("q", qkv[..., :NH, :], EPS / HD, s["q_scale"]), ("k", qkv[..., NH:NH + NKV, :], EPS, 1.0)):
        x = part.reshape(B, T * H * W, -1, HD).float()
        w = s[name + "_weight"]
        unit = x
        if s["norm"]:
            r = torch.rsqrt((x * x).mean(-1, keepdim=True) + eps)
            unit = x * r
        y = unit if w is None else unit * w.float()
        outs.append((_turn(y, cos, sin, s["interleaved"]) * scale).to(torch.bfloat16).reshape(part.shape))
        if s["op"] == "rope":
            continue
        g = _turn(s[f"d{name}_out"].reshape(x.shape).float(), cos, -sin, s["interleaved"]) * scale
        if not s["norm"]:
            grads.append(g.to(torch.bfloat16).reshape(part.shape))
            continue
        weights.append((g * unit).sum((0, 1, 2), dtype=torch.float64).float())
        g = g * w.float()
        dx = r * (g - unit * (g * unit).mean(-1, keepdim=True))
        grads.append(dx.to(torch.bfloat16).reshape(part.shape))
    return tuple(outs + grads + weights)


def _plain_cross(s):
    q, kv = s["q"], s["kv"]
    B, T, H, W, NH, HD = q.shape
    S, NKV = kv.shape[1], kv.shape[3]
    L, G = T * H * W, NH // NKV
    # a head of k and v and the rows of q that read it
    rows = lambda x: x.reshape(B, L, NKV, G, HD).permute(0, 2, 1, 3, 4).reshape(B, NKV, L * G, HD).float()  # noqa: E731
    back = lambda x: x.reshape(B, NKV, L, G, -1).permute(0, 2, 1, 3, 4).reshape(B, T, H, W, NH, -1)  # noqa: E731
    qs = rows(q)
    k, v = (kv[:, :, j].permute(0, 2, 1, 3).float() for j in range(2))
    p = qs @ k.transpose(-1, -2)                                   # (B, NKV, L*G, S)
    if s["kv_doc"] is not None:
        doc = s["doc"].reshape(B, L) if s["doc"] is not None else torch.zeros((B, L), dtype=torch.int32, device="cuda")
        unseen = (doc[:, :, None] != s["kv_doc"][:, None]) | (s["kv_doc"] < 0)[:, None]
        p.view(B, NKV, L, G, S).masked_fill_(unseen[:, None, :, None], -math.inf)
    top = p.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), 0.0, top)
    p = p.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    lse = back(top + torch.log(total)).squeeze(-1)
    p = p.div_(torch.where(total == 0, 1.0, total))
    out = p @ v
    result = back(out).to(torch.bfloat16)
    if s["op"] == "cross":
        return result, lse
    g = rows(s["dout"])
    dv = p.transpose(-1, -2) @ g
    ds = g @ v.transpose(-1, -2)
    ds = p * (ds - (p * ds).sum(-1, keepdim=True))
    dkv = torch.stack([ds.transpose(-1, -2) @ qs, dv], 2).permute(0, 3, 2, 1, 4)   # (B, S, 2, NKV, HD)
    return result, lse, back(ds @ k).to(torch.bfloat16), dkv.to(torch.bfloat16).contiguous()


def run(state):
    s = state
    if not own:
        return _plain_rope(s) if s["op"].startswith("rope") else _plain_cross(s)
    import neighborhood_attention_video_gb300 as na
    if s["op"].startswith("rope"):
        qkv, NH, NKV = s["qkv"], s["NH"], s["NKV"]
        HD = qkv.shape[-1]
        q, k = qkv[..., :NH, :], qkv[..., NH:NH + NKV, :]
        how = dict(q_weight=s["q_weight"], k_weight=s["k_weight"], table=s["table"], rope_dims=s["dims"], norm=s["norm"],
                   q_eps=EPS / HD, k_eps=EPS, q_scale=s["q_scale"], interleaved=s["interleaved"])
        q_out, k_out = (torch.empty(x.shape, dtype=x.dtype, device=x.device) for x in (q, k))
        na.na3d_norm_rope(q, k, q_out, k_out, **how)
        if s["op"] == "rope":
            return q_out, k_out
        dq, dk = torch.empty_like(q_out), torch.empty_like(k_out)
        dqw, dkw = (torch.empty(HD, device=qkv.device) for _ in range(2)) if s["norm"] else (None, None)
        na.na3d_norm_rope_bwd(q, k, s["dq_out"], s["dk_out"], dq, dk, dq_weight=dqw, dk_weight=dkw, **how)
        return (q_out, k_out, dq, dk, dqw, dkw) if s["norm"] else (q_out, k_out, dq, dk)
    k, v = s["kv"].unbind(2)
    docs = dict(doc=s["doc"], kv_doc=s["kv_doc"])
    out, lse = na.na3d_cross_attention(s["q"], k, v, return_lse=True, **docs)
    if s["op"] == "cross":
        return out, lse
    dq, dkv = torch.empty_like(s["q"]), torch.empty_like(s["kv"])
    na.na3d_cross_bwd(s["q"], k, v, out, lse, s["dout"], dq, *dkv.unbind(2), **docs)
    return out, lse, dq, dkv


def work(case):
    n = case["B"] * case["T"] * case["H"] * case["W"]
    NH, NKV, HD = case["NH"], case["NKV"], case["HD"]
    if case["op"].startswith("rope"):
        values = n * (NH + NKV) * HD
        table = 4 * (case["T"] * case["RT"] + case["H"] * case["RH"] + case["W"] * case["RW"]) + 4 * HD * case["norm"]
        if case["op"] == "rope":
            # squares and their sum, weight and norm, the rotation
            return {"bytes": 4 * values + table, "flops": 8 * values}
        # x read and the result written; x and the gradient read, its result written
        return {"bytes": 4 * values + (6 if case["norm"] else 4) * values + table, "flops": 24 * values}
    S, rows, states = case["S"], n * NH, case["B"] * case["S"] * NKV * HD
    # of packed clips a token reads its own clip's states alone
    pairs = rows * -(-S // max(1, case["docs"]))
    masks = (4 * n if case["docs"] else 0) + (4 * case["B"] * S if case["docs"] or case["pad"] else 0)
    # q, k and v read, out and lse written
    read_written = 4 * rows * HD + 4 * states + 4 * rows + masks
    if case["op"] == "cross":
        return {"bytes": read_written, "flops": 4 * pairs * HD}
    # q, k, v, out, dout and lse read again, dq, dk and dv written; the scores again, dp, dq, dk and dv
    return {"bytes": read_written + 8 * rows * HD + 8 * states + 4 * rows, "flops": 14 * pairs * HD}


# ------------------------------------------------------------------ 64 bits

def _exact_rope(case, s):
    """One frame after another, in 64 bits, the pairs as complex numbers."""
    f64, dev = torch.float64, "cuda"
    T, H, W, NH, NKV, HD = (case[n] for n in ("T", "H", "W", "NH", "NKV", "HD"))
    axis = [torch.repeat_interleave(torch.tensor([0, 1, 2], device=dev), torch.tensor([R // 2 for R in s["dims"]], device=dev)),
            torch.cat([torch.arange(R // 2, device=dev, dtype=f64) / (R // 2 or 1) for R in s["dims"]])]
    speed = torch.exp(-math.log(THETA) * axis[1])
    P = speed.numel()

    def split(x):
        if case["interleaved"]:
            z = torch.complex(x[..., 0:2 * P:2].contiguous(), x[..., 1:2 * P:2].contiguous())
        else:
            z = torch.complex(x[..., :P].contiguous(), x[..., P:2 * P].contiguous())
        return z, x[..., 2 * P:]

    def join(z, rest):
        flat = torch.view_as_real(z).flatten(-2) if case["interleaved"] else torch.cat([z.real, z.imag], -1)
        return torch.cat([flat, rest], -1)

    results = {n: [] for n in ("q", "k", "dq", "dk")}
    sums = {"q": torch.zeros(HD, dtype=f64, device=dev), "k": torch.zeros(HD, dtype=f64, device=dev)}
    for t in range(T):
        place = torch.stack([torch.full((H, W), t, device=dev), torch.arange(H, device=dev)[:, None].expand(H, W),
                             torch.arange(W, device=dev).expand(H, W)], -1).to(f64)
        angle = place[..., axis[0]] * speed                                  # (H, W, P)
        unit = torch.polar(torch.ones_like(angle), angle)[:, :, None]
        for name, lo, heads, eps, scale in (("q", 0, NH, EPS / HD, s["q_scale"]), ("k", NH, NKV, EPS, 1.0)):
            x = s["qkv"][:, t, :, :, lo:lo + heads].to(f64)
            w = torch.ones(HD, dtype=f64, device=dev) if s[name + "_weight"] is None else s[name + "_weight"].to(f64)
            size = torch.sqrt((x ** 2).sum(-1, keepdim=True) / HD + eps) if case["norm"] else torch.ones_like(x[..., :1])
            z, rest = split(x / size * w)
            results[name].append(scale * join(z * unit, rest))
            if case["op"] == "rope_train":
                z, rest = split(s[f"d{name}_out"][:, t].to(f64))
                g = scale * join(z * unit.conj(), rest)
                sums[name] += (g * x / size).sum((0, 1, 2, 3))
                g = g * w
                if case["norm"]:
                    g = (g - x * (g * x).sum(-1, keepdim=True) / (HD * size ** 2)) / size
                results["d" + name].append(g)
    order = ("q", "k") if case["op"] == "rope" else ("q", "k", "dq", "dk")
    got = [torch.stack(results[n], 1) for n in order]
    if case["op"] == "rope_train" and case["norm"]:
        got += [sums["q"], sums["k"]]
    return tuple(got)


def _exact_cross(case, s):
    """One entry and head of q after another, in 64 bits, over the states that each clip has."""
    f64 = torch.float64
    B, T, H, W, NH, HD, S, NKV = (case[n] for n in ("B", "T", "H", "W", "NH", "HD", "S", "NKV"))
    L, G, dev = T * H * W, NH // NKV, "cuda"
    out, lse = torch.zeros((B, L, NH, HD), dtype=f64, device=dev), torch.full((B, L, NH), -math.inf, dtype=f64, device=dev)
    train = case["op"] == "cross_train"
    dq, dkv = (torch.zeros_like(out), torch.zeros((B, S, 2, NKV, HD), dtype=f64, device=dev)) if train else (None, None)
    for b in range(B):
        doc = torch.zeros(L, device=dev) if s["doc"] is None else s["doc"][b].reshape(-1)
        kv_doc = torch.zeros(S, device=dev) if s["kv_doc"] is None else s["kv_doc"][b]
        for d in sorted(set(doc.tolist())):
            mine, theirs = torch.nonzero(doc == d)[:, 0], torch.nonzero(kv_doc == d)[:, 0]
            if d < 0 or not len(theirs):
                continue
            for n in range(NH):
                x = s["q"][b].reshape(L, NH, HD)[mine, n].to(f64)
                k, v = (s["kv"][b, theirs, j, n // G].to(f64) for j in range(2))
                logits = x @ k.t()
                total = torch.logsumexp(logits, 1)
                share = torch.exp(logits.sub_(total[:, None]))
                y = share @ v
                out[b, mine, n], lse[b, mine, n] = y, total
                if train:
                    g = s["dout"][b].reshape(L, NH, HD)[mine, n].to(f64)
                    slope = share * (g @ v.t() - (g * y).sum(1, keepdim=True))
                    dq[b, mine, n] = slope @ k
                    dkv[b, theirs, 0, n // G] += slope.t() @ x
                    dkv[b, theirs, 1, n // G] += share.t() @ g
    out, lse = out.view(B, T, H, W, NH, HD), lse.view(B, T, H, W, NH)
    return (out, lse, dq.view_as(out), dkv) if train else (out, lse)


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_rope(case, s) if case["op"].startswith("rope") else _exact_cross(case, s)
