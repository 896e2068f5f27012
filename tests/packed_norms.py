"""The score-shaped attention in 64 bits over whole rows of the score matrix, with
the expected square of each result's error: for windows so wide that the sum of
all roundings at their worst says nothing any more.

A rounding to bf16 is off by at most 2^-8 of the value, with a sign of its own:
the squares of that are summed where independent roundings meet in a sum, and
the square of the sum is taken where they share one (delta, in dq). Scores,
exponentials and fp32 sums count at 2^-16 of the magnitudes that enter, as in
the elementwise bounds. A result passes where the norm of its error is at most
twice the root of the summed squares.
"""
import math

import torch

import packed_reference as ref

F64 = torch.float64
HALF, FINE = ref.HALF, ref.FINE


def scored(q, k, v, g, kernel, softcap=0.0, slopes=None, doc=None, prefix=None, delta_by=1.0, cap_slope=True):
    """name -> (value, expected squared error), (B,T,H,W,NH,HD). delta_by and cap_slope
    spoil the gradients' formula: what a bound has to tell from the right one."""
    shape = q.shape
    B, T, H, W, NH, HD = shape
    n = T * H * W
    q, k, v, g = (x.detach().cpu().to(F64).reshape(B, n, NH, HD) for x in (q, k, v, g))
    seen = torch.zeros((n, n), dtype=torch.bool).scatter_(1, ref.window_index(T, H, W, kernel), True)
    pos = torch.stack([torch.arange(n) // (H * W), torch.arange(n) // W % H, torch.arange(n) % W])
    names = ("out", "dq", "dk", "dv")
    val, sq = ({name: torch.zeros_like(q) for name in names} for _ in range(2))
    for b in range(B):
        see = seen
        if doc is not None:
            d = doc[b].cpu().reshape(-1)
            see = see & (d[:, None] == d) & (d >= 0)
        if prefix is not None:
            see = see & ((pos[0] <= pos[0][:, None]) | (pos[0] < prefix[b].cpu()))
        for h in range(NH):
            x, y, z, w = (t[b, :, h] for t in (q, k, v, g))
            a, mag = x @ y.t(), x.abs() @ y.abs().t()
            th = torch.tanh(a / softcap) if softcap else torch.zeros_like(a)
            s = softcap * th if softcap else a
            if slopes is not None:
                far = sum(float(slopes[h, i]) * (pos[i] - pos[i][:, None]).abs().to(F64) for i in range(3))
                s, mag = s - far, mag + far.abs()
            s = s.masked_fill(~see, -math.inf)
            lse = torch.logsumexp(s, 1, keepdim=True)
            p = torch.where(see & torch.isfinite(lse), torch.exp(s - lse), 0.0)
            off = FINE * (1 + torch.where(see, mag, 0.0).amax(1, keepdim=True))      # of log p
            r2 = (HALF + 2 * off) ** 2
            out = p @ z
            out2 = r2 * (p ** 2 @ z ** 2) + HALF ** 2 * out ** 2
            dp, dpm = w @ z.t(), w.abs() @ z.abs().t()
            delta = (p * dp).sum(1, keepdim=True)
            cap = 1 - th * th if cap_slope else torch.ones_like(th)
            da = p * (dp - delta_by * delta) * cap
            pc = p * cap
            delta2 = (w ** 2 * out2).sum(1, keepdim=True)                      # dq: from the stored out
            exact2 = (2 * off * (p * dpm).sum(1, keepdim=True)) ** 2           # dk: the fp32 sum of p dp
            fine2 = ((2 * off + FINE) * pc * (dpm + delta.abs())) ** 2         # p and dp themselves
            dq, dk, dv = da @ y, da.t() @ x, p.t() @ w
            val["out"][b, :, h], sq["out"][b, :, h] = out, out2
            val["dq"][b, :, h] = dq
            sq["dq"][b, :, h] = delta2 * (pc @ y) ** 2 + (fine2 + FINE ** 2 * da ** 2) @ y ** 2 + HALF ** 2 * dq ** 2
            val["dk"][b, :, h] = dk
            sq["dk"][b, :, h] = (fine2 + HALF ** 2 * da ** 2 + exact2 * pc ** 2).t() @ x ** 2 + HALF ** 2 * dk ** 2
            val["dv"][b, :, h] = dv
            sq["dv"][b, :, h] = (r2 * p ** 2).t() @ w ** 2 + HALF ** 2 * dv ** 2
    return {name: (val[name].reshape(shape), sq[name].reshape(shape)) for name in names}


def excess(got, want):
    """The norm of the error over the largest that passes."""
    value, sq = want
    return float((got.detach().cpu().to(F64).reshape(value.shape) - value).norm() / (2 * sq.sum().sqrt()))
