"""Plain 64-bit forms of the attention's inputs (norms, rotation, paged-cache append) and of attention over a dequantised
cache, for the tests. Nothing here uses the package's kernels."""
from __future__ import annotations

import math

import torch

U32 = 2.0 ** -24                       # half a step of fp32, relative
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: U32}
F8 = torch.float8_e4m3fn
BLOCK = 32


def pairs(rot: int, interleaved: bool):
    i = torch.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def rotate(y, pos, inv_freq, interleaved, inverse=False):
    """y [B, N, H, d] fp64, pos [B, N] int64."""
    if inv_freq is None:
        return y.clone()
    a, b = pairs(2 * inv_freq.numel(), interleaved)
    t = pos.double()[..., None, None] * inv_freq.double()
    c, s = torch.cos(t), torch.sin(t)
    if inverse:
        s = -s
    z = y.clone()
    z[..., a] = y[..., a] * c - y[..., b] * s
    z[..., b] = y[..., a] * s + y[..., b] * c
    return z


def norm(x, w, eps):
    return x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w.double()


def forward(x, w, eps, pos, inv_freq, interleaved):
    return rotate(norm(x.double(), w, eps), pos, inv_freq, interleaved)


def forward_slack(x, w, eps, pos, inv_freq, interleaved):
    """fp32 error of a row's result before its last rounding: the mean of squares (12 roundings, halved by the root), rsqrt
    (2 steps), two products, cos and sin (an angle within 2^-24 turns: 6.3 steps, and 2 more), two products and a sum:
    under 32 half steps of |y_a| + |y_b|."""
    y = norm(x.double(), w, eps).abs()
    if inv_freq is None:
        return 32 * U32 * y
    a, b = pairs(2 * inv_freq.numel(), interleaved)
    m = y.clone()
    m[..., a] = m[..., b] = y[..., a] + y[..., b]
    return 32 * U32 * m


def backward(x, dz, w, eps, pos, inv_freq, interleaved):
    """(dx, dw, slack of dx, sum of |terms| of dw); dz [B, N, H, d]."""
    dz = dz.double()
    g = rotate(dz, pos, inv_freq, interleaved, inverse=True)
    mag = dz.abs()
    if inv_freq is not None:
        a, b = pairs(2 * inv_freq.numel(), interleaved)
        m = mag.clone()
        m[..., a] = m[..., b] = mag[..., a] + mag[..., b]
        mag = m
    if w is None:
        return g, None, 64 * U32 * mag, None
    x = x.double()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + eps)
    xh, wg = x * r, w.double() * g
    dx = r * (wg - xh * (wg * xh).mean(-1, keepdim=True))
    slack = 64 * U32 * r * (w.double().abs() * mag + xh.abs() * (w.double().abs() * mag * xh.abs()).mean(-1, keepdim=True))
    return dx, (g * xh).sum((0, 1, 2)), slack, (mag * xh.abs()).sum((0, 1, 2))


def need(amax):
    """Smallest power of two s with amax <= 448 s, in [2^-40, 2^40]."""
    e = torch.ceil(torch.log2(amax.double() / 448.0)).clamp(-40, 40)
    return torch.exp2(e.nan_to_num(neginf=-40.0))


def dequant(pages, scales):
    """[P, H, page, d] e4m3 and [P, H, page / 32] -> fp64."""
    P, H, page, d = pages.shape
    return (pages.float().double().view(P, H, page // BLOCK, BLOCK, d) * scales.double()[..., None, None]).view(P, H, page, d)


def gather(pages, table, n):
    """fp64 pages [P, H, page, d] and one request's ids -> [H, n, d]; a page that is not there reads as NaN."""
    P, H, page, d = pages.shape
    out = torch.full((H, n, d), math.nan, dtype=torch.float64)
    for c in range(-(-n // page)):
        if 0 <= int(table[c]) < P:
            m = min(page, n - c * page)
            out[:, c * page:c * page + m] = pages[int(table[c]), :, :m]
    return out


def attention(q, k, v, allowed, scale, slopes=None, pos=None, softcap=0.0, rel=None, kv_len=None):
    """One request, fp64: q [Hq, Q, d], k, v [Hkv, n, d], allowed [Q, n], pos [Q]. Returns O, LSE, and for the tolerances
    A = sum p |v| / sum p and the largest scale * sum_e |q_e k_e| of a row's visible pairs."""
    Hq, Q, d = q.shape
    g = Hq // k.shape[0]
    o, lse = torch.zeros_like(q), torch.full((Hq, Q), -math.inf, dtype=torch.float64)
    av, qk = torch.zeros_like(q), torch.zeros(Hq, Q, dtype=torch.float64)
    keep = allowed.any(0)
    if not keep.any():
        return o, lse, av, qk
    j = torch.nonzero(keep)[:, 0]
    al = allowed[:, j]
    for h in range(Hq):
        kk, vv = k[h // g, j], v[h // g, j]
        x = scale * q[h] @ kk.T
        dist = pos[:, None] - j[None]
        if slopes is not None:
            x = x - slopes[h].double() * dist
        if rel is not None:
            x = x + rel[h].double()[(dist + kv_len - 1).clamp(0, 2 * kv_len - 2)]
        if softcap:
            x = softcap * torch.tanh(x / softcap)
        x = x.masked_fill(~al, -math.inf)
        m = x.amax(-1, keepdim=True)
        p = torch.exp(x - torch.where(m.isinf(), torch.zeros_like(m), m))
        t = p.sum(-1, keepdim=True)
        live = t > 0
        p = p / torch.where(live, t, torch.ones_like(t))
        o[h], av[h] = p @ vv, p @ vv.abs()
        lse[h] = torch.where(live, m + torch.log(t), torch.full_like(t, -math.inf))[:, 0]
        qk[h] = scale * ((q[h].abs() @ kk.abs().T) * al).amax(-1)
    return o, lse, av, qk
