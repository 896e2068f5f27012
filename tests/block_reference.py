"""64-bit CPU references of the norm and rotation of queries and keys and of the
attention to states of another length, with elementwise error bounds.

A bound counts each rounding to bf16 at half a step (2^-8 of the value). The
attention's fp32 arithmetic (sums, exponentials, scores) counts at 2^-16 of the
magnitudes that enter, as for the windowed attention; the norm's and rotation's,
some ten operations and sums of up to 512 terms in a tree, at 2^-20.
"""
import math

import torch

F64 = torch.float64
HALF, FINE, ROPE_FINE = 2.0 ** -8, 2.0 ** -16, 2.0 ** -20


def angles(grid, dims, theta=10000.0, offset=(0, 0, 0), scale=(1, 1, 1)):
    """(T, H, W, P) angles of every position's pairs, the axes one behind another."""
    parts = []
    for a, (n, R) in enumerate(zip(grid, dims)):
        freq = torch.tensor([theta ** (-2.0 * i / R) for i in range(R // 2)], dtype=F64)
        ang = (offset[a] + scale[a] * torch.arange(n, dtype=F64))[:, None] * freq
        view = [1, 1, 1, R // 2]
        view[a] = n
        parts.append(ang.view(view).expand(*grid, R // 2))
    return torch.cat(parts, -1)


def table(grid, dims, **how):
    """The rows (cos, sin) in the layout of na3d_rope_table, in 64 bits."""
    rows = []
    for a, R in enumerate(dims):
        if R:
            index = [0, 0, 0]
            index[a] = slice(None)
            first = sum(dims[:a]) // 2
            ang = angles(grid, dims, **how)[tuple(index)][..., first:first + R // 2].reshape(-1)
            rows.append(torch.stack([ang.cos(), ang.sin()], -1))
    return torch.cat(rows)


def _turn(x, cos, sin, interleaved):
    """x (..., heads, HD) with its pairs turned, cos and sin (..., 1, P)."""
    P = cos.shape[-1]
    y = x.clone()
    i = torch.arange(P)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + P)
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def norm_rope(x, ang, weight=None, norm=True, eps=1e-6, scale=1.0, interleaved=True, dout=None):
    """out (and dx, dw) of one tensor (B, T, H, W, heads, HD), each with its bound.
    Rows of dout that are all zeros add nothing."""
    x = x.detach().cpu().to(F64)
    w = torch.ones(x.shape[-1], dtype=F64) if weight is None else weight.cpu().to(F64)
    cos, sin = ang.cos()[:, :, :, None], ang.sin()[:, :, :, None]
    live = torch.ones(x.shape[:-1] + (1,), dtype=torch.bool)
    if dout is not None:
        dout = dout.cpu().to(F64)
        live = (dout != 0).any(-1, keepdim=True)
    xs = torch.where(live, x, 0.0)
    got = {}
    r = 1 / torch.sqrt((xs ** 2).mean(-1, keepdim=True) + eps) if norm else torch.ones_like(xs[..., :1])
    full = x if dout is None else xs
    u = full * r
    y = _turn(u * w, cos, sin, interleaved) * scale
    mag = _turn((u * w).abs(), cos.abs(), -sin.abs(), interleaved)      # |a cos| + |b sin| for the first of a pair ...
    mag = torch.maximum(mag, _turn((u * w).abs(), cos.abs(), sin.abs(), interleaved)) * abs(scale)    # ... or the second
    got["out"] = (y, HALF * y.abs() + ROPE_FINE * mag + 1e-38)
    if dout is None:
        return got
    g = _turn(dout, cos, -sin, interleaved) * scale
    gm = torch.maximum(_turn(dout.abs(), cos.abs(), -sin.abs(), interleaved),
                       _turn(dout.abs(), cos.abs(), sin.abs(), interleaved)) * abs(scale)
    if not norm:
        got["dx"] = (g, HALF * g.abs() + ROPE_FINE * gm + 1e-38)
        return got
    got["dw"] = ((g * u).sum((0, 1, 2, 3, 4)), 8 * ROPE_FINE * (gm * u.abs()).sum((0, 1, 2, 3, 4)) + 1e-38)
    wg, wm = g * w, gm * w.abs()
    dx = torch.where(live, r * (wg - u * (wg * u).mean(-1, keepdim=True)), 0.0)
    dm = r * (wm + u.abs() * (wm * u.abs()).mean(-1, keepdim=True))
    got["dx"] = (dx, torch.where(live, HALF * dx.abs() + 4 * ROPE_FINE * dm + 1e-38, 0.0))
    return got


def cross(q, k, v, doc=None, kv_doc=None, dout=None):
    """out, lse (and dq, dk, dv) of q (B,T,H,W,NH,HD) and k, v (B,S,NKV,HD), each with
    its bound, one document and head after another: what it does not see is not in it."""
    B, T, H, W, NH, HD = q.shape
    S, NKV, L = k.shape[1], k.shape[2], T * H * W
    q, k, v = (x.detach().cpu().to(F64) for x in (q, k, v))
    doc = torch.zeros((B, L), dtype=torch.int64) if doc is None else doc.cpu().reshape(B, L).to(torch.int64)
    kv_doc = torch.zeros((B, S), dtype=torch.int64) if kv_doc is None else kv_doc.cpu().to(torch.int64)
    shape, states = (B, L, NH, HD), (B, S, NKV, HD)
    val, off = {}, {}
    for n, sh, fill in (("out", shape, 0.0), ("lse", shape[:3], -math.inf), ("dq", shape, 0.0), ("dk", states, 0.0), ("dv", states, 0.0)):
        val[n], off[n] = torch.full(sh, fill, dtype=F64), torch.zeros(sh, dtype=F64)
    qf = q.reshape(shape)
    gf = None if dout is None else dout.detach().cpu().to(F64).reshape(shape)
    for b in range(B):
        for d in set(doc[b].tolist()):
            i, j = torch.nonzero(doc[b] == d)[:, 0], torch.nonzero(kv_doc[b] == d)[:, 0]
            if d < 0 or not len(j):
                continue
            for h in range(NH):
                c = h // (NH // NKV)
                x, y, z = qf[b, i, h], k[b, j, c], v[b, j, c]
                s = x @ y.t()
                fine = FINE * (1 + (x.abs() @ y.abs().t()).amax(1, keepdim=True))      # of a score, and so of log p
                lse = torch.logsumexp(s, 1, keepdim=True)
                p = torch.exp(s - lse)
                out, vm = p @ z, p @ z.abs()
                o_off = HALF * (out.abs() + vm) + 2 * fine * vm
                val["out"][b, i, h], off["out"][b, i, h] = out, o_off
                val["lse"][b, i, h], off["lse"][b, i, h] = lse[:, 0], fine[:, 0] / 8
                if gf is None:
                    continue
                g = gf[b, i, h]
                dp, dpm = g @ z.t(), g.abs() @ z.abs().t()
                delta = (p * dp).sum(1, keepdim=True)
                # delta may come from the stored out: its rounding, and that of the probabilities in it
                d_off = (g.abs() * o_off).sum(1, keepdim=True)
                ds = p * (dp - delta)
                s_off = p * d_off + HALF * ds.abs() + 4 * fine * p * (dpm + delta.abs())
                p_off = (HALF + 2 * fine) * p
                val["dq"][b, i, h], off["dq"][b, i, h] = ds @ y, s_off @ y.abs()
                val["dk"][b, j, c] += ds.t() @ x
                off["dk"][b, j, c] += s_off.t() @ x.abs()
                val["dv"][b, j, c] += p.t() @ g
                off["dv"][b, j, c] += p_off.t() @ g.abs()
    got = {"out": (val["out"].view(q.shape), off["out"].view(q.shape)), "lse": (val["lse"].view(q.shape[:5]), off["lse"].view(q.shape[:5]))}
    if gf is not None:
        for n in ("dq", "dk", "dv"):
            e = off[n] + HALF * (val[n].abs() + off[n])
            e = torch.where(e > 0, e + 1e-30, e)
            got[n] = (val[n].view(q.shape if n == "dq" else states), e.view(q.shape if n == "dq" else states))
    return got
