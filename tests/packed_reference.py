"""64-bit CPU references of the packed-batch operators (attention with shaped
scores, projection with adapters), with elementwise error bounds.

A bound counts each rounding to bf16 at half a step (2^-8 of the value) and the
fp32 arithmetic of sums, exponentials and scores at 2^-16 of the magnitudes
that enter (2^-24 for each operation, with room for sums of up to 256 terms in
sequence; longer sums are split).
"""
import math

import torch

F64 = torch.float64
HALF, FINE = 2.0 ** -8, 2.0 ** -16


def window_index(T, H, W, kernel):
    axes = []
    for n, k in zip((T, H, W), kernel):
        i = torch.arange(n)
        start = (i - k // 2).clamp(min=0).clamp(max=n - k)
        axes.append(start[:, None] + torch.arange(k)[None])
    t, h, w = axes
    idx = (t[:, None, None, :, None, None] * H + h[None, :, None, None, :, None]) * W + w[None, None, :, None, None, :]
    return idx.reshape(T * H * W, -1)


def scored(q, k, v, kernel, softcap=0.0, slopes=None, doc=None, prefix=None, dout=None, given=None):
    """out, lse (and dq, dk, dv) of (B,T,H,W,NH,HD) inputs in 64 bits, each with
    its bound: a dict name -> (value, bound). Masked keys are taken as zeros
    before any product. given: (out, lse) of the forward pass for the backward
    pass's delta; the exact ones where it is None."""
    B, T, H, W, NH, HD = q.shape
    n = T * H * W
    q, k, v = (x.detach().cpu().to(F64).reshape(B, n, NH, HD) for x in (q, k, v))
    idx = window_index(T, H, W, kernel)
    seen = torch.ones((B, n, idx.shape[1]), dtype=torch.bool)
    if doc is not None:
        d = doc.cpu().reshape(B, n)
        seen &= (d[:, idx] == d[:, :, None]) & (d[:, :, None] >= 0)
    if prefix is not None:
        frame = torch.arange(n) // (H * W)
        seen &= (frame[idx] <= frame[:, None])[None] | (frame[idx][None] < prefix.cpu()[:, None, None])
    sees = seen.any(-1)                                            # (B, n)
    qs = torch.where(sees[..., None, None], q, 0.0)
    kw = torch.where(seen[..., None, None], k[:, idx], 0.0)        # (B, n, keys, NH, HD)
    vw = torch.where(seen[..., None, None], v[:, idx], 0.0)
    a = torch.einsum("bnhd,bnkhd->bnkh", qs, kw)
    mag = torch.einsum("bnhd,bnkhd->bnkh", qs.abs(), kw.abs())
    th = torch.tanh(a / softcap) if softcap else torch.zeros_like(a)
    s = softcap * th if softcap else a
    if slopes is not None:
        pos = torch.stack([torch.arange(n) // (H * W), torch.arange(n) // W % H, torch.arange(n) % W], -1)
        far = (pos[idx] - pos[:, None]).abs().to(F64) @ slopes.cpu().to(F64).t()
        s, mag = s - far, mag + far.abs()
    s = s.masked_fill(~seen[..., None], -math.inf)
    lse = torch.logsumexp(s, 2)
    p = torch.where(seen[..., None], torch.exp(s - lse[:, :, None]), 0.0)
    out = torch.einsum("bnkh,bnkhd->bnhd", p, vw)
    vmag = torch.einsum("bnkh,bnkhd->bnhd", p, vw.abs())
    off = FINE * (1 + mag.amax(2))                                  # of a score, and so of log p
    full = (B, T, H, W, NH, HD)
    got = {"out": (out.reshape(full), (HALF * (out.abs() + vmag) + 2 * off[..., None] * vmag).reshape(full)),
           "lse": (lse.reshape(full[:5]), (off / 8).reshape(full[:5]))}
    if dout is None:
        return got
    g = torch.where(sees[..., None, None], dout.cpu().to(F64).reshape(B, n, NH, HD), 0.0)
    dp = torch.einsum("bnhd,bnkhd->bnkh", g, vw)
    delta = (p * dp).sum(2)
    # delta from the stored out: its rounding, and that of the probabilities in it
    d_off = torch.einsum("bnhd,bnhd->bnh", g.abs(), HALF * (out.abs() + vmag) + 2 * off[..., None] * vmag)
    cap = 1 - th * th
    da = p * (dp - delta[:, :, None]) * cap
    dpm = torch.einsum("bnhd,bnkhd->bnkh", g.abs(), vw.abs())
    da_off = p * d_off[:, :, None] + HALF * da.abs() + 4 * off[:, :, None] * p * (dpm + delta[:, :, None].abs())
    p_off = (HALF + 2 * off[:, :, None]) * p

    def scatter(x):
        return torch.zeros_like(k).index_add_(1, idx.reshape(-1), x.reshape(B, -1, NH, HD))

    def rounded(x, e):
        return x.reshape(full), (e + HALF * (x.abs() + e) + 1e-30).reshape(full)

    got["dq"] = rounded(torch.einsum("bnkh,bnkhd->bnhd", da, kw), torch.einsum("bnkh,bnkhd->bnhd", da_off, kw.abs()))
    got["dk"] = rounded(scatter(da[..., None] * qs[:, :, None]), scatter(da_off[..., None] * qs[:, :, None].abs()))
    got["dv"] = rounded(scatter(p[..., None] * g[:, :, None]), scatter(p_off[..., None] * g[:, :, None].abs()))
    return got


def row_adapters(offsets, adapter, n_adapters, M):
    """The adapter of every row, -1 for none."""
    of = torch.full((M,), -1, dtype=torch.int64)
    for r, a in enumerate(adapter.tolist()):
        if 0 <= a < n_adapters:
            of[int(offsets[r]):int(offsets[r + 1])] = a
    return of


def lora(x, w, bias, lora_a, lora_b, scaling, offsets, adapter, HD, dqkv=None):
    """qkv (and dx, da, db) in 64 bits with bounds: a dict name -> (value, bound)."""
    x, w, a, b, sc = (t.detach().cpu().to(F64) for t in (x, w, lora_a, lora_b, scaling))
    M, N, n_ad = x.shape[0], w.shape[0], a.shape[0]
    of = row_adapters(offsets.cpu(), adapter.cpu(), n_ad, M)
    s = torch.ones(N, dtype=F64)
    s[:N // 3] = HD ** -0.5
    y, mag = x @ w.t(), x.abs() @ w.abs().t()
    t, tm = torch.zeros((M, a.shape[1]), dtype=F64), torch.zeros((M, a.shape[1]), dtype=F64)
    tb = torch.zeros_like(y)
    for i in range(n_ad):
        rows = of == i
        t[rows], tm[rows] = sc[i] * (x[rows] @ a[i].t()), sc[i].abs() * (x[rows].abs() @ a[i].abs().t())
        y[rows] += t[rows] @ b[i].t()
        tb[rows] = t[rows].abs() @ b[i].abs().t()
        mag[rows] += tm[rows] @ b[i].abs().t()
    if bias is not None:
        y, mag = y + bias.cpu().to(F64), mag + bias.cpu().to(F64).abs()
    e = (HALF * tb + FINE * mag) * s
    y = y * s
    got = {"qkv": (y, e + HALF * (y.abs() + e) + 1e-30)}
    if dqkv is None:
        return got
    g = dqkv.cpu().to(F64).reshape(M, N) * s
    dx, dxm = g @ w, g.abs() @ w.abs()
    da, dam, db, dbm = (torch.zeros_like(z) for z in (a, a, b, b))
    dxe, dae, dbe = torch.zeros_like(dx), torch.zeros_like(a), torch.zeros_like(b)
    for i in range(n_ad):
        rows = of == i
        u, um = sc[i] * (g[rows] @ b[i]), sc[i].abs() * (g[rows].abs() @ b[i].abs())
        dx[rows] += u @ a[i]
        dxm[rows] += um @ a[i].abs()
        dxe[rows] = HALF * (u.abs() @ a[i].abs())
        da[i], dam[i], dae[i] = u.t() @ x[rows], um.t() @ x[rows].abs(), HALF * (u.abs().t() @ x[rows].abs())
        db[i], dbm[i], dbe[i] = g[rows].t() @ t[rows], g[rows].abs().t() @ tm[rows], HALF * (g[rows].abs().t() @ t[rows].abs())
    for name, val, m, err in (("dx", dx, dxm, dxe), ("da", da, dam, dae), ("db", db, dbm, dbe)):
        err = err + FINE * m
        got[name] = (val, err + HALF * (val.abs() + err) + 1e-30)
    return got


def check(name, got, want):
    """Every value within its bound; infinities equal."""
    value, bound = want
    got = got.detach().cpu().to(F64).reshape(value.shape)
    inf = torch.isinf(value)
    assert torch.equal(torch.isinf(got), inf) and torch.equal(got[inf], value[inf]), f"{name}: infinities differ"
    err = (got - value).abs()[~inf]
    assert torch.isfinite(err).all(), f"{name}: NaN"
    over = err > bound[~inf]          # a bound of 0 (a row that sees nothing) wants the value itself
    if bool(over.any()):
        ratio = float((err / bound[~inf].clamp(min=1e-300))[over].max())
        raise AssertionError(f"{name}: {int(over.sum())} values off, up to {ratio:.3f} times their bound")
