"""Plain 64-bit forms of the key-block bounds and of the choice of blocks, for the tests."""
import numpy as np
import torch

F8 = torch.float8_e4m3fn


def key_bounds(k, Bk):
    """[B, H, nk, 2, d] doubles of keys [B, H, N, d]; NaN stays."""
    k = k.double().cpu()
    out = []
    for x in k.split(Bk, 2):
        out.append(torch.stack([x.amin(2), x.amax(2)], 2))
    return torch.stack(out, 2)


def scores(q, box):
    """sum over queries [n, d] and channels of max(q min, q max), per block of box [nk, 2, d]: numpy doubles."""
    with np.errstate(invalid="ignore", over="ignore"):
        pos, neg = np.where(q > 0, q, 0.0).sum(0), np.where(q > 0, 0.0, q).sum(0)
        return (pos * box[:, 1]).sum(1) + (neg * box[:, 0]).sum(1)


def choose(cls, score, keep, first, last):
    """Columns kept of one row: classes [nk], scores [nk]. NaN ranks above everything, ties go to the lower column."""
    cand = np.flatnonzero(cls)
    if len(cand) <= keep:
        return set(cand.tolist())
    ends = set(cand[:first].tolist()) | set(cand[len(cand) - last:].tolist())
    rest = [c for c in cand.tolist() if c not in ends]
    rest.sort(key=lambda c: (0 if np.isnan(score[c]) else 1, 0.0 if np.isnan(score[c]) else -score[c], c))
    return ends | set(rest[:keep - first - last])


def select(src_class, q, box, keep, first, last, bq):
    """Classes [B, Hkv, nq, nk] of the mask that is chosen. src_class [Bm, 1, nq, nk]; q [B, Hq, Q, d]; box(b, hk) -> [nk, 2, d] doubles,
    with -inf scores for rows of None."""
    B, Hq, Q, d = q.shape
    q = q.double().cpu().numpy()
    src = src_class.cpu().numpy()
    nq, nk = src.shape[2:]
    Hkv = box.heads
    out = np.zeros((B, Hkv, nq, nk), np.uint8)
    for b in range(B):
        for h in range(Hkv):
            bx, gone = box(b, h)
            for r in range(nq):
                g = Hq // Hkv
                rows = q[b, h * g:(h + 1) * g, r * bq:(r + 1) * bq].reshape(-1, d)
                s = scores(rows, bx)
                s[gone] = -np.inf
                c = src[b if src.shape[0] > 1 else 0, 0, r]
                kept = choose(c, s, keep, first, last)
                for j in kept:
                    out[b, h, r, j] = c[j]
    return out


class Dense:
    def __init__(self, bounds):
        self.x, self.heads = bounds.double().cpu().numpy(), bounds.shape[1]

    def __call__(self, b, h):
        return self.x[b, h], np.zeros(self.x.shape[2], bool)


class Paged:
    def __init__(self, bounds, table, nk):
        self.x, self.heads = bounds.double().cpu().numpy(), bounds.shape[1]
        self.t = table.cpu().numpy()[:, :nk]

    def __call__(self, b, h):
        bad = (self.t[b] < 0) | (self.t[b] >= len(self.x))
        return self.x[np.where(bad, 0, self.t[b]), h], bad


def tables(cls):
    """The tables of a mask with these classes, as the builder lays them out."""
    B, H, nq, nk = cls.shape
    out = dict(block_class=cls)
    for name, kind in (("kv", 1), ("full_kv", 2)):
        num, idx = np.zeros((B, H, nq), np.int32), np.zeros((B, H, nq, nk), np.int32)
        tnum, tidx = np.zeros((B, H, nk), np.int32), np.zeros((B, H, nk, nq), np.int32)
        for b in range(B):
            for h in range(H):
                for r in range(nq):
                    c = np.flatnonzero(cls[b, h, r] == kind)
                    num[b, h, r], idx[b, h, r, :len(c)] = len(c), c
                for j in range(nk):
                    c = np.flatnonzero(cls[b, h, :, j] == kind)
                    tnum[b, h, j], tidx[b, h, j, :len(c)] = len(c), c
        t = "full_q" if kind == 2 else "q"
        out |= {name + "_num": num, name + "_idx": idx, t + "_num": tnum, t + "_idx": tidx}
    if nq > 1:
        ln = out["kv_num"] + out["full_kv_num"]
        desc = np.arange(nq - 1, -1, -1)
        order = np.broadcast_to(desc, (B, H, nq)) if nk > 2048 else desc[np.argsort(-ln[..., desc], axis=-1, kind="stable")]
        out["row_order"] = order.astype(np.int32)
    return out


def allowed(cls, pairs, bq, bk):
    """Pairs [.., Q, N] of the rule that lie in visited blocks, per (b, h): cls [B, H, nq, nk], pairs [B or 1, Q, N] -> [B, H, Q, N]."""
    Q, N = pairs.shape[-2:]
    vis = np.repeat(np.repeat(cls > 0, bq, 2)[:, :, :Q], bk, 3)[..., :N]
    return vis & pairs[:, None]


def attention(q, k, v, ok, scale, softcap=0.0, dout=None):
    """O, LSE (and dQ, dK, dV) in doubles: q [B, Hq, Q, d], k, v [B, Hkv, N, d], ok [B, Hkv, Q, N] truth values."""
    B, Hq, Q, d = q.shape
    g = Hq // k.shape[1]
    q, k, v = (x.double().cpu() for x in (q, k, v))
    ke, ve = k.repeat_interleave(g, 1), v.repeat_interleave(g, 1)
    ok = torch.as_tensor(ok).repeat_interleave(g, 1)
    s = q @ ke.transpose(-1, -2) * scale
    if softcap:
        t = torch.tanh(s / softcap)
        s = softcap * t
    s = s.masked_fill(~ok, -torch.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse.nan_to_num(neginf=0.0)[..., None])
    o = p @ ve
    if dout is None:
        return o, lse
    do = dout.double().cpu()
    ds = p * (do @ ve.transpose(-1, -2) - (do * o).sum(-1, keepdim=True))
    if softcap:
        ds = ds * (1 - t * t)
    fold = lambda x: x.view(B, -1, g, *x.shape[2:]).sum(2)  # noqa: E731
    return o, lse, ds @ ke * scale, fold(ds.transpose(-1, -2) @ q * scale), fold(p.transpose(-1, -2) @ do)
