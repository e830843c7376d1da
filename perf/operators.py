"""Cases for the operators around the attention's inputs and its 8-bit paged cache.

  rope_forward / rope_backward   norms of the query and key heads, position rotation, and the move from the projections' token-major
                                 rows to the head-major tensors the attention reads (and its gradient)
  append                         one step's keys and values into the paged cache (bf16, or e4m3 with a power-of-two scale for each
                                 32 tokens and head), normalised and rotated on the way, and the step's queries
  decode                         one query token per request over the 8-bit paged cache
  prefill                        a chunk of query tokens per request over the 8-bit paged cache

A pass returns whole outputs. The cache's pages are float8 tensors: their values and their scales are returned side by side."""
import math

import torch

own = False

BLOCK = 32                      # tokens that share a scale
F8 = torch.float8_e4m3fn
F8_MAX = 448.0
SCALE_LO, SCALE_HI = 2.0 ** -40, 2.0 ** 40


# ---------------------------------------------------------------------------------------------- cases
def listed():
    rope = dict(eps=1e-6, theta=10000.0, norm=True, interleaved=False)
    cache = dict(window=0, prefix=0, softcap=0.0, alibi=False)
    return [
        # the causal training workload's projections on their way into the attention
        dict(name="rope forward 4x4096", op="rope_forward", B=4, N=4096, Hq=16, Hkv=16, d=128, rot=128, offset=0, **rope),
        # the packed-document workload's gradients on their way back to the projections
        dict(name="rope backward 16384", op="rope_backward", B=1, N=16384, Hq=32, Hkv=8, d=128, rot=128, offset=0, **rope),
        # a small batch of odd length, partial rotation in neighbouring pairs, far positions
        dict(name="rope backward 3x333", op="rope_backward", B=3, N=333, Hq=4, Hkv=2, d=64, rot=32, offset=900001, eps=1e-5,
             theta=500000.0, norm=True, interleaved=True),
        # a decode step of 64 requests: one token each, bf16 cache
        dict(name="append 64x1 bf16", op="append", fp8=False, B=64, N=1, Hq=32, Hkv=8, d=128, rot=128, page=128, context=2000, ragged=False, **rope),
        # the same step into the 8-bit cache: most tokens continue a block
        dict(name="append 64x1 fp8", op="append", fp8=True, B=64, N=1, Hq=32, Hkv=8, d=128, rot=128, page=128, context=2000, ragged=False, **rope),
        # prompt chunks of a padded batch into the 8-bit cache
        dict(name="append 8x2048 fp8", op="append", fp8=True, B=8, N=2048, Hq=32, Hkv=8, d=128, rot=128, page=128, context=1000, ragged=True, **rope),
        # one short request: the latency of a single call
        dict(name="decode 1x500", op="decode", B=1, lo=500, hi=500, Hq=4, Hkv=2, d=64, page=32, window=128, prefix=0, softcap=20.0, alibi=False),
        # the paged decode workload over the 8-bit cache
        dict(name="decode 64x1k-32k", op="decode", B=64, lo=1024, hi=32768, Hq=32, Hkv=8, d=128, page=128, **cache),
        # two long requests: few rows, a long axis
        dict(name="decode 2x131072", op="decode", B=2, lo=120000, hi=131072, Hq=32, Hkv=8, d=128, page=64, **cache),
        # a short prompt chunk of several requests with windowed, soft-capped scores
        dict(name="prefill 3x100", op="prefill", B=3, Q=100, lo=300, hi=1000, Hq=4, Hkv=2, d=64, page=64, window=128, prefix=0, softcap=20.0, alibi=False),
        # chunked prefill at the end of a long context
        dict(name="prefill 256 of 131072", op="prefill", B=1, Q=256, lo=131072, hi=131072, Hq=8, Hkv=8, d=128, page=128, **cache),
        # a batch of chunks, grouped heads, ALiBi
        dict(name="prefill 4x1024 of 4096", op="prefill", B=4, Q=1024, lo=2048, hi=4096, Hq=32, Hkv=8, d=128, page=128, window=0, prefix=0, softcap=0.0, alibi=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope_forward", "rope_backward", "append", "append", "decode", "decode", "prefill"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 8])
    rope = dict(rot=16 * rng.randint(1, d // 16), eps=rng.choice([1e-6, 1e-5]), theta=rng.choice([10000.0, 500000.0]), norm=rng.random() < 0.8,
                interleaved=rng.random() < 0.3)
    rules = dict(window=rng.choice([0, 0, _log(rng, 1, 4000)]), prefix=0, softcap=rng.choice([0.0, 0.0, 20.0, 50.0]), alibi=False)
    if rules["softcap"] == 0.0:
        rules["alibi"] = rng.random() < 0.3
    if rules["window"] == 0 and rng.random() < 0.3:
        rules["prefix"] = _log(rng, 1, 500)
    page = rng.choice([32, 64, 128])
    if op.startswith("rope"):
        B = rng.randint(1, 4)
        return dict(op=op, B=B, N=_log(rng, 1, 4 * 4096 * 48 // (B * (Hq + 2 * Hkv))) if Hq + 2 * Hkv > 48 else _log(rng, 1, 16384 // B), Hq=Hq,
                    Hkv=Hkv, d=d, offset=rng.choice([0, _log(rng, 1, 1000000)]), **rope)
    if op == "append":
        B = _log(rng, 1, 64)
        return dict(op=op, fp8=rng.random() < 0.7, B=B, N=_log(rng, 1, max(1, 16384 // B)) if rng.random() < 0.6 else 1, Hq=Hq, Hkv=Hkv, d=d, page=page,
                    context=_log(rng, 1, 2000), ragged=rng.random() < 0.5, **rope)
    if op == "decode":
        B = _log(rng, 1, 64)
        hi = _log(rng, 1, min(131072, 2 ** 20 // B))
        return dict(op=op, B=B, lo=max(1, hi // rng.choice([1, 4, 32])), hi=hi, Hq=Hq, Hkv=Hkv, d=d, page=page, **rules)
    B, Q = rng.randint(1, 4), _log(rng, 1, 1024)
    hi = Q + _log(rng, 1, max(1, min(131072, 2 ** 28 // (B * Q * Hq)) - Q))
    return dict(op=op, B=B, Q=Q, lo=max(Q, hi // rng.choice([1, 4])), hi=hi, Hq=Hq, Hkv=Hkv, d=d, page=page, **rules)


# ---------------------------------------------------------------------------------------------- inputs
def _quantised(g, P, Hkv, page, d):
    """A pool of e4m3 pages that an appending program has left: N(0, 1) values with a few strong channels, in blocks of 32 tokens."""
    channel = 1 + 7 * (torch.rand(d, generator=g, device="cuda") > 0.95)
    pages = torch.empty(P, Hkv, page, d, dtype=F8, device="cuda")
    scales = torch.empty(P, Hkv, page // BLOCK, dtype=torch.float32, device="cuda")
    step = max(1, (1 << 26) // (Hkv * page * d))
    for p in range(0, P, step):
        x = torch.randn(min(step, P - p), Hkv, page // BLOCK, BLOCK, d, generator=g, device="cuda") * channel
        s = torch.exp2(torch.ceil(torch.log2(x.abs().amax((-1, -2)) / F8_MAX)))
        pages[p:p + step] = (x / s[..., None, None]).to(F8).view(-1, Hkv, page, d)
        scales[p:p + step] = s
    return pages, scales


def _table(g, lens, page, width, total=None):
    """Pages of each request at shuffled ids, -1 behind them, and the size of the pool: some pages belong to nobody."""
    need = (lens + page - 1) // page
    total = total or int(need.sum()) + 3
    ids = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    at = torch.arange(width, device="cuda")[None]
    first = torch.cumsum(need, 0) - need
    return torch.where(at < need[:, None], ids[(first[:, None] + at).clamp(max=total - 1)], torch.full_like(ids[:1], -1)), total


def _lengths(g, B, lo, hi):
    lens = torch.randint(lo, hi + 1, (B,), generator=g, device="cuda")
    lens[0] = hi
    return lens


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, Hq, Hkv, d, op = case["B"], case["Hq"], case["Hkv"], case["d"], case["op"]
    s = dict(case=case)
    if op in ("rope_forward", "rope_backward", "append"):
        N, H = case["N"], Hq + 2 * Hkv
        channel = 1 + 7 * (torch.rand(H, d, generator=g, device="cuda") > 0.95)
        s["qkv"] = (torch.randn(B, N, H, d, generator=g, device="cuda") * channel).to(torch.bfloat16)  # the packed projection's output
        s["wq"] = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")) if case["norm"] else None
        s["wk"] = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")) if case["norm"] else None
        s["inv_freq"] = case["theta"] ** (-2 * torch.arange(case["rot"] // 2, device="cuda", dtype=torch.float64) / case["rot"])
        s["inv_freq"] = s["inv_freq"].to(torch.float32)
        if op == "append":
            offset = _lengths(g, B, 0, case["context"])
            n_new = torch.randint(N // 2, N + 1, (B,), generator=g, device="cuda") if case["ragged"] else torch.full((B,), N, device="cuda")
            width = (case["context"] + N + case["page"] - 1) // case["page"]
            s["table"], total = _table(g, offset + n_new, case["page"], width, B * width + 3)
            s["n_new"] = n_new.to(torch.int32)
            if case["fp8"]:
                s["k"], s["ks"] = _quantised(g, total, Hkv, case["page"], d)
                s["v"], s["vs"] = _quantised(g, total, Hkv, case["page"], d)
            else:
                s["k"], s["v"] = (torch.randn(total, Hkv, case["page"], d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
            s["q_out"] = torch.zeros(B, Hq, N, d, dtype=torch.bfloat16, device="cuda")
        else:
            offset = torch.full((B,), case["offset"], device="cuda") + torch.randint(0, 100, (B,), generator=g, device="cuda")
        s["offset"] = offset.to(torch.int32)
        if op == "rope_backward":
            s["dq"], s["dk"], s["dv"] = (torch.randn(B, h, N, d, generator=g, device="cuda") for h in (Hq, Hkv, Hkv))
    else:
        Q = case.get("Q", 1)
        lens = _lengths(g, B, case["lo"], case["hi"])
        width = (case["hi"] + case["page"] - 1) // case["page"]
        s["table"], total = _table(g, lens, case["page"], width)
        s["k"], s["ks"] = _quantised(g, total, Hkv, case["page"], d)
        s["v"], s["vs"] = _quantised(g, total, Hkv, case["page"], d)
        s["q"] = torch.randn(B, Hq, Q, d, generator=g, device="cuda").to(torch.bfloat16)
        s["offset"] = (lens - Q).to(torch.int32)
        s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, Hq + 1, device="cuda", dtype=torch.float32) / Hq) if case["alibi"] else None
    if own:
        _handles(s)
    return s


def _handles(s):
    """What a serving or training program holds across calls: the rules, one mask for all layers of a step, a workspace, the status word."""
    from block_sparse_masked_create_gb300 import fa
    c = s["case"]
    if "qkv" in s:
        s["rule"] = fa.make_qk_rule(s["wq"], s["wk"], c["eps"], s["inv_freq"], interleaved=c["interleaved"])
        return
    spec = [("causal",)]
    if c["window"]:
        spec += [("window", c["window"]), ("and",)]
    if c["prefix"]:
        spec += [("prefix", c["prefix"]), ("or",)]
    rule = fa.make_mask_rule(spec, q_offset=s["offset"], batch_dependent=True)
    # a prefix is shown to every row, also where it is longer than a request: those positions name page 0, as in the plain form
    s["pages"] = s["table"].clamp(min=0)
    s["capacity"] = s["table"].shape[1] * c["page"]
    if c["op"] == "decode":
        s["mask"] = fa.create_block_mask(rule, c["B"], c["Hq"], 1, s["capacity"], 1, c["page"], keep=[s["offset"]])
    else:
        s["mask"] = fa.create_block_mask(rule, c["B"], c["Hq"], c["Q"], s["capacity"], 128, 128, keep=[s["offset"]])
    s["score"] = fa.make_score_rule(s["slopes"], softcap=c["softcap"])


# ---------------------------------------------------------------------------------------------- a pass
def run(s):
    if own:
        return _own(s)
    op = s["case"]["op"]
    if op == "rope_forward":
        return tuple(x.transpose(1, 2).contiguous() for x in _rows(s))
    if op == "rope_backward":
        return _rows_backward(s)
    return _append(s) if op == "append" else _attend(s)


def _own(s):
    from block_sparse_masked_create_gb300 import fa
    c, op = s["case"], s["case"]["op"]
    if "qkv" in s:
        q, k, v = s["qkv"].split([c["Hq"], c["Hkv"], c["Hkv"]], dim=2)
        if op == "rope_forward":
            return fa.qk_norm_rope(q, k, v, s["rule"], q_offset=s["offset"])
        if op == "rope_backward":
            grad = torch.empty_like(s["qkv"])
            dq, dk, dv = grad.split([c["Hq"], c["Hkv"], c["Hkv"]], dim=2)
            dwq, dwk = fa.qk_norm_rope_backward(q, k, s["dq"], s["dk"], s["dv"], s["rule"], q_offset=s["offset"], dq_in=dq, dk_in=dk, dv_in=dv)[3:]
            return (grad, dwq, dwk) if c["norm"] else (grad,)
        if not c["fp8"]:
            fa.kv_append(q, k, v, s["k"], s["v"], s["table"], s["rule"], q_offset=s["offset"], n_new=s["n_new"], q_out=s["q_out"])
            return s["q_out"], s["k"], s["v"]
        fa.kv_append_fp8(q, k, v, s["k"], s["v"], s["ks"], s["vs"], s["table"], s["rule"], q_offset=s["offset"], n_new=s["n_new"], q_out=s["q_out"])
        return s["q_out"], s["k"], s["ks"], s["v"], s["vs"]
    if op == "decode":
        o, lse = fa.flex_decode_fp8(s["q"][:, :, 0], s["k"], s["v"], s["ks"], s["vs"], s["pages"], s["mask"], s["score"])
        return o[:, :, None], lse[..., None]
    return fa.flex_forward_paged_fp8(s["q"], s["k"], s["v"], s["ks"], s["vs"], s["pages"], s["mask"], s["capacity"], s["score"])


def _angles(s):
    """cos and sin of each token's rotation [B, N, 1, rot / 2]; the angles of far positions need 64 bits."""
    at = s["offset"].double()[:, None] + torch.arange(s["case"]["N"], device="cuda")
    a = at[..., None, None] * s["inv_freq"].double()
    return torch.cos(a).float(), torch.sin(a).float()


def _pairs(x, c):
    """The two halves of each rotated pair, and the rest of the row."""
    r = c["rot"]
    if c["interleaved"]:
        return x[..., 0:r:2], x[..., 1:r:2], x[..., r:]
    return x[..., :r // 2], x[..., r // 2:r], x[..., r:]


def _unpairs(a, b, rest, c):
    if c["interleaved"]:
        return torch.cat([torch.stack([a, b], -1).flatten(-2), rest], -1)
    return torch.cat([a, b, rest], -1)


def _rows(s, dtype=torch.bfloat16):
    """q, k, v [B, N, H, d], the first two normalised and rotated."""
    c = s["case"]
    cos, sin = _angles(s)
    q, k, v = s["qkv"].split([c["Hq"], c["Hkv"], c["Hkv"]], dim=2)

    def one(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + c["eps"]) * w
        a, b, rest = _pairs(x, c)
        return _unpairs(a * cos - b * sin, a * sin + b * cos, rest, c).to(dtype)

    return one(q, s["wq"]), one(k, s["wk"]), v.to(dtype)


def _rows_backward(s):
    c = s["case"]
    cos, sin = _angles(s)
    q, k, _ = s["qkv"].split([c["Hq"], c["Hkv"], c["Hkv"]], dim=2)

    def one(x, dy, w):
        a, b, rest = _pairs(dy.transpose(1, 2), c)
        g = _unpairs(a * cos + b * sin, b * cos - a * sin, rest, c)
        if w is None:
            return g, None
        x = x.float()
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + c["eps"])
        xh, wg = x * r, w * g
        return r * (wg - xh * (wg * xh).mean(-1, keepdim=True)), (g * xh).double().sum((0, 1, 2)).float()

    dq, dwq = one(q, s["dq"], s["wq"])
    dk, dwk = one(k, s["dk"], s["wk"])
    grad = torch.cat([dq, dk, s["dv"].transpose(1, 2)], 2).to(torch.bfloat16)
    return (grad, dwq, dwk) if c["norm"] else (grad,)


def _append(s):
    c = s["case"]
    B, N, page, d, Hkv = c["B"], c["N"], c["page"], c["d"], c["Hkv"]
    q, k, v = _rows(s, torch.float32)
    live = torch.arange(N, device="cuda")[None] < s["n_new"][:, None]
    s["q_out"].copy_(torch.where(live[:, None, :, None], q.transpose(1, 2).to(torch.bfloat16), s["q_out"]))
    first, last = s["offset"].long(), (s["offset"] + s["n_new"]).long()
    if not c["fp8"]:
        at = first[:, None] + torch.arange(N, device="cuda")
        pid = torch.gather(s["table"].long(), 1, (at // page).clamp(max=s["table"].shape[1] - 1))[live]
        slot = (at % page)[live]
        s["k"][pid, :, slot] = k[live].to(torch.bfloat16)
        s["v"][pid, :, slot] = v[live].to(torch.bfloat16)
        return s["q_out"], s["k"], s["v"]
    # the 32-token blocks that each request's new tokens reach: [B, blocks, 32] positions
    blocks = first[:, None] // BLOCK + torch.arange((N + 2 * BLOCK - 2) // BLOCK, device="cuda")
    touched = blocks * BLOCK < last[:, None]
    at = blocks[..., None] * BLOCK + torch.arange(BLOCK, device="cuda")
    new = (at >= first[:, None, None]) & (at < last[:, None, None])
    old = at < first[:, None, None]
    pid = torch.gather(s["table"].long(), 1, (blocks * BLOCK // page).clamp(max=s["table"].shape[1] - 1))[touched]
    sub = (blocks % (page // BLOCK))[touched]
    b = torch.arange(B, device="cuda")[:, None].expand_as(blocks)[touched]
    at, new, old = at[touched], new[touched], old[touched]
    for x, pages, scales in ((k, s["k"], s["ks"]), (v, s["v"], s["vs"])):
        n = (at - first[b][:, None]).clamp(0, N - 1)
        fresh = x[b[:, None], n].transpose(1, 2)                                    # [T, Hkv, 32, d]
        need = torch.where(new[:, None, :, None], fresh.abs(), 0).amax((-1, -2))
        frac, e = torch.frexp(need / F8_MAX)                                        # smallest power of two >= need / 448
        need = torch.ldexp(torch.ones_like(need), torch.where(frac == 0.5, e - 1, e)).where(need > 0, 0).clamp(SCALE_LO, SCALE_HI)
        before = scales[pid, :, sub]
        after = torch.where(old[:, :1], torch.maximum(before, need), need)
        view = pages.view(pages.shape[0], Hkv, page // BLOCK, BLOCK, d)
        was = view.view(torch.uint8)[pid, :, sub]
        kept = (was.view(F8).float() * (before / after)[..., None, None]).to(F8).view(torch.uint8)
        now = (fresh / after[..., None, None]).clamp(-F8_MAX, F8_MAX).to(F8).view(torch.uint8)
        view.view(torch.uint8)[pid, :, sub] = torch.where(new[:, None, :, None], now, torch.where(old[:, None, :, None], kept, was))
        scales[pid, :, sub] = after
    return s["q_out"], s["k"], s["ks"], s["v"], s["vs"]


def _attend(s):
    c = s["case"]
    B, Hq, Hkv, d, page, Q = c["B"], c["Hq"], c["Hkv"], c["d"], c["page"], c.get("Q", 1)
    ids = s["table"].clamp(min=0).long()
    n = ids.shape[1] * page

    def gather(pages, scales):
        x = pages.view(torch.uint8)[ids].view(F8).float().view(B, -1, Hkv, page // BLOCK, BLOCK, d) * scales[ids][..., None, None]
        return x.view(B, -1, Hkv, page, d).transpose(1, 2).reshape(B, Hkv, n, d)

    i = s["offset"].long()[:, None] + torch.arange(Q, device="cuda")
    gap = i[:, :, None] - torch.arange(n, device="cuda")                             # i - j [B, Q, n]
    seen = gap >= 0
    if c["window"]:
        seen &= gap < c["window"]
    if c["prefix"]:
        seen |= (torch.arange(n, device="cuda") < c["prefix"])[None, None]
    k, v = gather(s["k"], s["ks"]), gather(s["v"], s["vs"])
    x = torch.matmul(s["q"].float().view(B, Hkv, -1, d), k.transpose(-1, -2)).view(B, Hq, Q, n) / math.sqrt(d)
    if s["slopes"] is not None:
        x -= s["slopes"][:, None, None] * gap[:, None]
    if c["softcap"]:
        x = c["softcap"] * torch.tanh(x / c["softcap"])
    x.masked_fill_(~seen[:, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m.isinf(), 0, m))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Hkv, -1, n), v).view(B, Hq, Q, d) / torch.where(total == 0, 1, total)
    return o.to(torch.bfloat16), (m + torch.log(total)).squeeze(-1)


# ---------------------------------------------------------------------------------------------- work
def work(case):
    c = case
    B, Hq, Hkv, d, op = c["B"], c["Hq"], c["Hkv"], c["d"], c["op"]
    if op in ("rope_forward", "rope_backward"):
        rows = B * c["N"]
        if op == "rope_forward":                            # bf16 in, bf16 out; norm 4, rotation 3 operations a value
            return dict(bytes=rows * (Hq + 2 * Hkv) * d * 4, flops=rows * (Hq + Hkv) * d * 7)
        read = (Hq + Hkv) * d * (6 if c["norm"] else 4) + Hkv * d * 4
        return dict(bytes=rows * (read + (Hq + 2 * Hkv) * d * 2), flops=rows * (Hq + Hkv) * d * 16)
    if op == "append":
        rows = B * c["N"] * (0.75 if c["ragged"] and c["N"] > 1 else 1)
        out = Hq * d * 2 + 2 * Hkv * d * (1 if c["fp8"] else 2)
        return dict(bytes=rows * ((Hq + 2 * Hkv) * d * 2 + out), flops=rows * (Hq + Hkv) * d * 7)
    mean = (c["lo"] + c["hi"]) / 2 if B > 1 else c["hi"]
    Q = c.get("Q", 1)
    reach = lambda n: min(n, c["window"]) if c["window"] else n                      # noqa: E731
    tokens = B * min(mean, reach(mean) + Q)
    pairs = B * Hq * Q * reach(max(1.0, mean - (Q - 1) / 2))
    return dict(bytes=tokens * Hkv * (d + 4 / BLOCK) * 2 + B * Hq * Q * (4 * d + 4), flops=4 * d * pairs)


# ---------------------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    """The definition in 64 bits, a request (and a head) at a time. Values that a cache holds are given as they are before they are rounded."""
    s = prepare(case, seed)
    c, op = case, case["op"]
    B, Hq, Hkv, d = c["B"], c["Hq"], c["Hkv"], c["d"]
    if op in ("decode", "prefill"):
        return _exact_attention(s)
    N, r = c["N"], c["rot"]
    first = (torch.arange(r // 2) * 2 if c["interleaved"] else torch.arange(r // 2)).cuda()
    second = first + (1 if c["interleaved"] else r // 2)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       (s["offset"].double()[:, None] + torch.arange(N, device="cuda"))[..., None] * s["inv_freq"].double())
    heads, grads, dw = [], [], {"q": 0, "k": 0}
    for h in range(Hq + 2 * Hkv):
        x = s["qkv"][:, :, h].double()
        kind = "q" if h < Hq else "k" if h < Hq + Hkv else "v"
        w = None if kind == "v" or not c["norm"] else s["w" + kind].double()
        norm = (x.pow(2).sum(-1, keepdim=True) / d + c["eps"]).sqrt()
        if op == "rope_backward":
            g = s["d" + kind][:, h - {"q": 0, "k": Hq, "v": Hq + Hkv}[kind]].double()
            if kind != "v":
                z = torch.complex(g[..., first], g[..., second]) * turn.conj()
                g[..., first], g[..., second] = z.real, z.imag
            if w is not None:
                dw[kind] = dw[kind] + (g * x / norm).sum((0, 1))
                g = w * g / norm - x * ((w * g * x).sum(-1, keepdim=True) / (d * norm.pow(3)))
            grads.append(g)
            continue
        if w is not None:
            x = x / norm * w
        if kind != "v":
            z = torch.complex(x[..., first], x[..., second]) * turn
            x[..., first], x[..., second] = z.real, z.imag
        heads.append(x)
    if op == "rope_backward":
        return (torch.stack(grads, 2), dw["q"], dw["k"]) if c["norm"] else (torch.stack(grads, 2),)
    q, k, v = torch.stack(heads[:Hq], 1), torch.stack(heads[Hq:Hq + Hkv], 1), torch.stack(heads[Hq + Hkv:], 1)
    if op == "rope_forward":
        return q, k, v
    page, table = c["page"], s["table"].tolist()
    q_out = s["q_out"].double()
    pools = [s["k"].double(), s["v"].double()]
    scales = [s["ks"].double(), s["vs"].double()] if c["fp8"] else None
    for b, (lo, n) in enumerate(zip(s["offset"].tolist(), s["n_new"].tolist())):
        q_out[b, :, :n] = q[b, :, :n]
        step = BLOCK if c["fp8"] else page
        for at in range(lo - lo % step, lo + n, step):
            i, j = max(at, lo), min(at + step, lo + n)
            if j <= i:
                continue
            pid, slot, keep = table[b][at // page], at % page, i - at
            for z in range(2):
                x = (k, v)[z][b, :, i - lo:j - lo]
                if not c["fp8"]:
                    pools[z][pid, :, slot + keep:slot + j - at] = x
                    continue
                need = 2.0 ** torch.ceil(torch.log2(x.abs().amax((1, 2)) / F8_MAX)).clamp(-40, 40)
                was = scales[z][pid, :, slot // BLOCK].clone()
                now = torch.maximum(need, was) if keep else need
                scales[z][pid, :, slot // BLOCK] = now
                pools[z][pid, :, slot:slot + keep] *= (was / now)[:, None, None]
                pools[z][pid, :, slot + keep:slot + j - at] = (x / now[:, None, None]).clamp(-F8_MAX, F8_MAX)
    return (q_out, pools[0], scales[0], pools[1], scales[1]) if c["fp8"] else (q_out, pools[0], pools[1])


def _exact_attention(s):
    c = s["case"]
    B, Hq, Hkv, d, page, Q = c["B"], c["Hq"], c["Hkv"], c["d"], c["page"], c.get("Q", 1)
    out = torch.zeros(B, Hq, Q, d, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq, Q), -math.inf, dtype=torch.float64, device="cuda")
    for b, lo in enumerate(s["offset"].tolist()):
        n = lo + Q
        ids = s["table"][b, :(n + page - 1) // page].long()
        i, j = lo + torch.arange(Q, device="cuda")[:, None], torch.arange(n, device="cuda")[None]
        hidden = j > i
        if c["window"]:
            hidden = hidden | (i - j >= c["window"])
        if c["prefix"]:
            hidden = hidden & (j >= c["prefix"])
        for h in range(Hkv):
            k, v = (p[ids, h].double().view(-1, BLOCK, d).mul(t[ids, h].double().view(-1, 1, 1)).view(-1, d)[:n] for p, t in ((s["k"], s["ks"]), (s["v"], s["vs"])))
            for hq in range(h * (Hq // Hkv), (h + 1) * (Hq // Hkv)):
                x = s["q"][b, hq].double() @ k.T * d ** -0.5
                if s["slopes"] is not None:
                    x = x - s["slopes"][hq].double() * (i - j)
                if c["softcap"]:
                    x = torch.tanh(x / c["softcap"]) * c["softcap"]
                x = x.masked_fill(hidden, -math.inf)
                z = torch.logsumexp(x, -1)
                lse[b, hq] = z
                out[b, hq] = torch.exp(x - z[:, None].nan_to_num(neginf=0.0)) @ v
    return out, lse
