"""Cases for attention over the key blocks that a cheap score picks for each query block.

  bounds   the smallest and the largest key of each block, channel by channel: of a whole tensor of keys, or of the pages of a cache
           that a step's tokens reach (bf16, or e4m3 with a scale for each 32 tokens)
  choose   for each query block and KV head, the `keep` blocks of a mask's row with the largest bound on <q, k>, summed over the block's
           queries and the heads of the group; the first and the last few of the row always: the tables of the smaller mask
  decode   one query token per request over the pages chosen for each KV head, bf16 or 8-bit cache
  step     a decode step: bounds of the newest page, choice, attention
  train    a training step: bounds, choice, forward and backward

The score of block c for a query q is  sum_e max(q_e min_e(c), q_e max_e(c)),  an upper bound of <q, k> over the block's keys k. It is
compared in 64 bits: neighbours in rank can lie closer than 32 bits tell apart."""
import math

import torch

own = False

BLOCK = 32                      # tokens that share a scale in the 8-bit cache
F8 = torch.float8_e4m3fn
F8_MAX = 448.0


# ---------------------------------------------------------------------------------------------- cases
def listed():
    serve = dict(Hq=32, Hkv=8, d=128, first=1, last=2, window=0, softcap=0.0)
    rows = dict(lo=0, paged=False, first=1, last=1)
    return [
        # a decode step of 64 requests: the page that the newest token lies in
        dict(name="bounds 64x1 bf16", op="bounds", kind="bf16", B=64, N=1, Hkv=8, d=128, block=64, context=4000, ragged=False),
        # prompt chunks of a padded batch in the 8-bit cache
        dict(name="bounds 8x2048 fp8", op="bounds", kind="fp8", B=8, N=2048, Hkv=8, d=128, block=128, context=1000, ragged=True),
        # the keys of the causal training workload
        dict(name="bounds 4x4096", op="bounds", kind="dense", B=4, N=4096, Hkv=16, d=128, block=128, context=0, ragged=False),
        # one short request with a window: the latency of a single call
        dict(name="choose 1x600", op="choose", B=1, Q=1, lo=600, hi=600, Hq=4, Hkv=2, d=64, block=32, keep=8, first=1, last=2, window=400, paged=True),
        # the paged decode workload: a step's choice of 2048 tokens for each request and KV head
        dict(name="choose 64x1k-32k", op="choose", B=64, Q=1, lo=1024, hi=32768, Hq=32, Hkv=8, d=128, block=64, keep=32, first=1, last=2, window=0, paged=True),
        # two long requests: few rows, a long axis
        dict(name="choose 2x131072", op="choose", B=2, Q=1, lo=120000, hi=131072, Hq=32, Hkv=8, d=128, block=64, keep=64, first=1, last=2, window=0, paged=True),
        # the causal training workload's query blocks
        dict(name="choose 4x4096 rows", op="choose", B=4, Q=4096, hi=4096, Hq=16, Hkv=16, d=128, block=128, keep=8, window=0, **rows),
        # a long sequence's query blocks, grouped heads
        dict(name="choose 65536 rows", op="choose", B=1, Q=65536, hi=65536, Hq=16, Hkv=4, d=128, block=128, keep=32, window=0, **rows),
        # attention of the paged decode workload over what was chosen
        dict(name="decode 64x1k-32k", op="decode", fp8=False, B=64, lo=1024, hi=32768, block=64, keep=32, **serve),
        # the same of two long requests over the 8-bit cache
        dict(name="decode 2x131072 fp8", op="decode", fp8=True, B=2, lo=120000, hi=131072, block=64, keep=64, **serve),
        # a whole decode step over the 8-bit cache
        dict(name="step 64x1k-32k fp8", op="step", fp8=True, B=64, lo=1024, hi=32768, block=64, keep=32, **serve),
        # a training step over a long sequence
        dict(name="train 8192", op="train", B=1, Q=8192, hi=8192, Hq=16, Hkv=4, d=128, block=128, keep=16, window=0, **rows),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["bounds", "bounds", "choose", "choose", "choose", "decode", "decode", "step", "train"])
    d, block = rng.choice([64, 128]), rng.choice([32, 64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    if op == "bounds":
        kind = rng.choice(["dense", "bf16", "fp8"])
        B = rng.randint(1, 4) if kind == "dense" else _log(rng, 1, 64)
        N = _log(rng, 1, 4 * 4096 * 16 // (B * Hkv)) if kind == "dense" else _log(rng, 1, max(1, 16384 // B)) if rng.random() < 0.5 else 1
        return dict(op=op, kind=kind, B=B, N=N, Hkv=Hkv, d=d, block=block, context=0 if kind == "dense" else _log(rng, 1, 8000),
                    ragged=kind != "dense" and rng.random() < 0.5)
    Hq = Hkv * rng.choice([1, 2, 3, 4, 8])
    window = rng.choice([0, 0, _log(rng, 1, 20000)])
    first, last = rng.randint(0, 2), rng.randint(1, 3)
    keep = first + last + _log(rng, 1, 64) - 1
    least = 1
    if op == "choose":  # blocks enough for a choice: its outputs are nothing else
        least = (first + last + 24) * max(block, 64)
        window = window and max(window, least)
        keep = first + last + rng.randint(1, 12)
    if op == "train" or op == "choose" and rng.random() < 0.5:
        # query blocks of a training batch, or of a chunk over a cache
        block = 128 if op == "train" else max(block, 64)
        paged = op == "choose" and rng.random() < 0.4
        B = rng.randint(1, 3)
        if op == "train":
            Hq = min(Hq, 2 * Hkv)
            Q = _log(rng, 1, 8192 // B)
        else:
            Q = _log(rng, 1, 2048) if paged else _log(rng, least, 65536 * 16 // (B * max(16, Hq)) * block // 128)
        hi = Q + _log(rng, 2 * least, 60000) if paged else Q
        return dict(op=op, B=B, Q=Q, lo=max(Q, hi // 2) if paged else 0, hi=hi, Hq=Hq, Hkv=Hkv, d=d, block=block, keep=keep, first=first, last=last,
                    window=window, paged=paged)
    B = _log(rng, 1, 64)
    hi = _log(rng, least, min(131072, 2 ** 20 // B))
    case = dict(op=op, B=B, lo=max(1, hi // rng.choice([1, 4, 32])), hi=hi, Hq=Hq, Hkv=Hkv, d=d, block=block, keep=keep, first=first, last=last, window=window)
    if op == "choose":
        return dict(case, Q=1, paged=True)
    return dict(case, fp8=rng.random() < 0.5, softcap=rng.choice([0.0, 0.0, 20.0]))


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


def _pool(s, g, P, names):
    c = s["case"]
    shape = (P, c["Hkv"], c["block"], c["d"])
    for x in names:
        if c.get("fp8") or c.get("kind") == "fp8":
            s[x], s[x + "s"] = _quantised(g, *shape)
        else:
            s[x] = torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g)


def _table(g, lens, page, width):
    """Pages of each request at shuffled ids, -1 behind them, and the size of the pool: some pages belong to nobody."""
    need = (lens + page - 1) // page
    total = len(lens) * width + 3
    ids = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    at = torch.arange(width, device="cuda")[None]
    first = torch.cumsum(need, 0) - need
    return torch.where(at < need[:, None], ids[(first[:, None] + at).clamp(max=total - 1)], torch.full_like(ids[:1], -1)), total


def _lengths(g, B, lo, hi):
    lens = torch.randint(lo, hi + 1, (B,), generator=g, device="cuda")
    lens[0] = hi
    return lens


def _bounds(g, n, Hkv, d):
    """Bounds of blocks that an earlier step has left, [n, Hkv, 2, d]: each block's keys lie about a centre of its own, a few channels are strong."""
    channel = 1 + 7 * (torch.rand(Hkv, d, generator=g, device="cuda") > 0.95)
    centre = 0.5 * torch.randn(n, Hkv, d, generator=g, device="cuda")
    half = 1.5 + torch.rand(n, Hkv, 2, d, generator=g, device="cuda")
    half[:, :, 0] *= -1
    return ((centre[:, :, None] + half) * channel[:, None]).to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c, op = case, case["op"]
    B, Hkv, d, block = c["B"], c["Hkv"], c["d"], c["block"]
    s = dict(case=c)
    if op == "bounds" and c["kind"] == "dense":
        s["k"] = torch.randn(B, Hkv, c["N"], d, generator=g, device="cuda").to(torch.bfloat16)
        return s
    if op == "bounds":
        N = c["N"]
        offset = _lengths(g, B, 0, c["context"])
        s["n_new"] = (torch.randint(N // 2, N + 1, (B,), generator=g, device="cuda") if c["ragged"] else torch.full((B,), N, device="cuda")).to(torch.int32)
        s["offset"] = offset.to(torch.int32)
        s["table"], total = _table(g, offset + s["n_new"], block, (c["context"] + N + block - 1) // block)
        _pool(s, g, total, "k")
        s["bounds"] = _bounds(g, total, Hkv, d)
        return s
    Hq, Q = c["Hq"], c.get("Q", 1)
    s["q"] = torch.randn(B, Hq, Q, d, generator=g, device="cuda").to(torch.bfloat16)
    if op == "train":
        s["k"], s["v"] = (torch.randn(B, Hkv, Q, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
        s["dout"] = torch.randn(B, Hq, Q, d, generator=g, device="cuda").to(torch.bfloat16)
    elif op == "choose" and not c["paged"]:
        s["bounds"] = _bounds(g, B * ((Q + block - 1) // block), Hkv, d).view(B, -1, Hkv, 2, d).transpose(1, 2).contiguous()
    else:
        lens = _lengths(g, B, c["lo"], c["hi"])
        s["offset"] = (lens - Q).to(torch.int32)
        s["table"], total = _table(g, lens, block, (c["hi"] + block - 1) // block)
        s["bounds"] = _bounds(g, total, Hkv, d)
        if op != "choose":
            _pool(s, g, total, "kv")
        if op == "decode" and not own:
            s["chosen"] = _choose(s)[0]
    if own:
        _handles(s)
    return s


def _handles(s):
    """What a program keeps across the layers of a step: the mask of its rule, and for the attention alone the mask that was chosen from it."""
    from block_sparse_masked_create_gb300 import fa
    c = s["case"]
    spec = [("causal",)] + ([("window", c["window"]), ("and",)] if c["window"] else [])
    rule = fa.make_mask_rule(spec, q_offset=s.get("offset"))
    Q, block = c.get("Q", 1), c["block"]
    n = s["table"].shape[1] * block if "table" in s else Q
    s["mask"] = fa.create_block_mask(rule, c["B"], c["Hq"], Q, n, 1 if Q == 1 and "table" in s else block, block)
    s["score"] = fa.make_score_rule(softcap=c.get("softcap", 0.0))
    if c["op"] == "decode":
        s["mask"] = fa.select_blocks(s["mask"], s["q"], s["bounds"], c["keep"], c["first"], c["last"], page_table=s["table"])


# ---------------------------------------------------------------------------------------------- a pass
def run(s):
    if own:
        return _own(s)
    c, op = s["case"], s["case"]["op"]
    if op == "bounds":
        return _block_bounds(s["k"], c["block"]) if c["kind"] == "dense" else _page_bounds(s)
    if op == "choose":
        return _tables(*_choose(s))
    if op == "decode":
        return _attend(s, s["chosen"])
    if op == "step":
        bounds = _page_bounds(s)
        return (bounds, *_attend(s, _choose(s)[0]))
    return _train(s)


def _own(s):
    from block_sparse_masked_create_gb300 import fa
    c, op = s["case"], s["case"]["op"]
    if op == "bounds":
        if c["kind"] == "dense":
            return fa.key_bounds(s["k"], c["block"])
        if c["kind"] == "fp8":
            return fa.kv_bounds_fp8(s["k"], s["ks"], s["bounds"], s["table"], c["N"], q_offset=s["offset"], n_new=s["n_new"])
        return fa.kv_bounds(s["k"], s["bounds"], s["table"], c["N"], q_offset=s["offset"], n_new=s["n_new"])
    pick = dict(keep=c["keep"], first=c["first"], last=c["last"], page_table=s.get("table"))
    if op == "choose":
        return fa.select_blocks(s["mask"], s["q"], s["bounds"], **pick).tables()
    if op == "train":
        bounds = fa.key_bounds(s["k"], c["block"])
        mask = fa.select_blocks(s["mask"], s["q"], bounds, **pick)
        o, lse = fa.flex_forward(s["q"], s["k"], s["v"], mask)
        grads = fa.flex_backward(s["q"], s["k"], s["v"], o, lse, s["dout"], mask)
        return (o, lse, *(x.to(torch.bfloat16) for x in grads))
    mask, out = s["mask"], ()
    if op == "step":
        if c["fp8"]:
            out = (fa.kv_bounds_fp8(s["k"], s["ks"], s["bounds"], s["table"], 1, q_offset=s["offset"]),)
        else:
            out = (fa.kv_bounds(s["k"], s["bounds"], s["table"], 1, q_offset=s["offset"]),)
        mask = fa.select_blocks(mask, s["q"], s["bounds"], **pick)
    q = s["q"][:, :, 0]
    if c["fp8"]:
        return (*out, *fa.flex_decode_fp8(q, s["k"], s["v"], s["ks"], s["vs"], s["table"], mask, s["score"]))
    return (*out, *fa.flex_decode(q, s["k"], s["v"], s["table"], mask, s["score"]))


def _block_bounds(k, block):
    """[B, Hkv, blocks, 2, d] of keys [B, Hkv, N, d]."""
    B, H, N, d = k.shape
    pad = -N % block
    x = k.float()
    lo = torch.nn.functional.pad(x, (0, 0, 0, pad), value=math.inf).view(B, H, -1, block, d).amin(3)
    hi = torch.nn.functional.pad(x, (0, 0, 0, pad), value=-math.inf).view(B, H, -1, block, d).amax(3)
    return torch.stack([lo, hi], 3).to(torch.bfloat16)


def _page_bounds(s):
    """Bounds of the pages that the newest tokens reach, over each page's tokens up to the last of them; other pages' stay."""
    c = s["case"]
    N, page = c.get("N", 1), c["block"]
    first = s["offset"].long()
    last = first + (s["n_new"].long() if "n_new" in s else N)
    at = first[:, None] // page + torch.arange((N + 2 * page - 2) // page, device="cuda")
    reached = (at * page < last[:, None]) & (last > first)[:, None]
    pid = torch.gather(s["table"].long(), 1, at.clamp(max=s["table"].shape[1] - 1))[reached]
    held = (last[:, None] - at * page).clamp(max=page)[reached]
    if "ks" in s:
        x = s["k"].view(torch.uint8)[pid].view(F8).float().view(-1, c["Hkv"], page // BLOCK, BLOCK, c["d"]) * s["ks"][pid][..., None, None]
        x = x.view(-1, c["Hkv"], page, c["d"])
    else:
        x = s["k"][pid].float()
    live = (torch.arange(page, device="cuda") < held[:, None])[:, None, :, None]
    s["bounds"][pid] = torch.stack([x.masked_fill(~live, math.inf).amin(2), x.masked_fill(~live, -math.inf).amax(2)], 2).to(torch.bfloat16)
    return s["bounds"]


def _classes(s):
    """0 empty, 1 partial, 2 full: the class of each (query block, key block) of the causal rule [B, nq, nk]."""
    c = s["case"]
    Q, bk = c.get("Q", 1), c["block"]
    paged = "table" in s
    bq = 1 if Q == 1 and paged else bk
    n = s["table"].shape[1] * bk if paged else Q
    i0 = torch.arange(0, Q, bq, device="cuda")[None, :, None] + (s["offset"].long()[:, None, None] if paged else torch.zeros(c["B"], 1, 1, dtype=torch.long, device="cuda"))
    rows = (Q - torch.arange(0, Q, bq, device="cuda")).clamp(max=bq)[None, :, None]
    j0 = torch.arange(0, n, bk, device="cuda")[None, None]
    cols = (n - j0).clamp(max=bk)
    least, most = i0 - (j0 + cols - 1), i0 + rows - 1 - j0
    window = c["window"] or 1 << 40
    some = (most >= 0) & (least < window)
    every = (least >= 0) & (most < window) & (rows == bq) & (cols == bk)
    return some.to(torch.uint8) + every.to(torch.uint8)


def _block_of(s):
    """The bounds of each request's blocks [B, Hkv, nk, 2, d]."""
    if "table" not in s:
        return s["bounds"]
    return s["bounds"][s["table"].clamp(min=0).long()].transpose(1, 2)


def _choose(s):
    """Which blocks of each (request, KV head, query block) are kept [B, Hkv, nq, nk], and the classes they are chosen from."""
    c = s["case"]
    B, Hq, Hkv, d = c["B"], c["Hq"], c["Hkv"], c["d"]
    kinds = _classes(s)
    nq = kinds.shape[1]
    bq = c["block"] if nq > 1 or "table" not in s else c.get("Q", 1)
    q = torch.nn.functional.pad(s["q"], (0, 0, 0, nq * bq - s["q"].shape[2])).view(B, Hkv, Hq // Hkv, nq, bq, d).double()
    box = _block_of(s).double()
    score = q.clamp(min=0).sum((2, 4)) @ box[:, :, :, 1].transpose(-1, -2) + q.clamp(max=0).sum((2, 4)) @ box[:, :, :, 0].transpose(-1, -2)
    seen = (kinds > 0)[:, None]
    rank = torch.cumsum(seen, -1) - 1
    count = seen.sum(-1, keepdim=True)
    always = seen & ((rank < c["first"]) | (rank >= count - c["last"]))
    score = score.masked_fill(always | ~seen, -math.inf)
    order = torch.argsort(score, dim=-1, descending=True, stable=True)
    place = torch.empty_like(order).scatter_(-1, order, torch.arange(order.shape[-1], device="cuda").expand_as(order))
    return always | seen & ~always & (place < c["keep"] - always.sum(-1, keepdim=True)), kinds


def _lists(x):
    """Counts of a truth table's rows, and its columns in ascending order with zeros behind them."""
    n = x.shape[-1]
    at = torch.arange(n, device="cuda", dtype=torch.int32)
    num = x.sum(-1, dtype=torch.int32)
    idx = torch.sort(torch.where(x, at, n), dim=-1).values.to(torch.int32)
    return num, torch.where(at < num[..., None], idx, 0)


def _tables(chosen, kinds):
    kinds = torch.where(chosen, kinds[:, None], torch.zeros_like(kinds[:, None]))
    part, full = kinds == 1, kinds == 2
    lists = [_lists(x) for x in (part, full, part.transpose(-1, -2), full.transpose(-1, -2))]
    names = ("kv_num", "full_kv_num", "q_num", "full_q_num", "kv_idx", "full_kv_idx", "q_idx", "full_q_idx")
    out = dict(zip(names, [x for x, _ in lists] + [x for _, x in lists]), block_class=kinds)
    nq = kinds.shape[2]
    if nq > 1:  # rows by length from the longest, of equal ones the later first
        key = (out["kv_num"] + out["full_kv_num"]).long() * nq + torch.arange(nq, device="cuda")
        out["row_order"] = torch.argsort(key, dim=-1, descending=True).to(torch.int32)
    return out


def _attend(s, chosen):
    """One query token per request over its chosen pages: O bf16 [B, Hq, d], LSE [B, Hq]."""
    c = s["case"]
    B, Hq, Hkv, d, page = c["B"], c["Hq"], c["Hkv"], c["d"], c["block"]
    ids = s["table"].clamp(min=0).long()
    n = ids.shape[1] * page

    def gather(x):
        if c["fp8"]:
            y = s[x].view(torch.uint8)[ids].view(F8).float().view(B, -1, Hkv, page // BLOCK, BLOCK, d) * s[x + "s"][ids][..., None, None]
            return y.view(B, -1, Hkv, page, d).transpose(1, 2).reshape(B, Hkv, n, d)
        return s[x][ids].transpose(1, 2).reshape(B, Hkv, n, d).float()

    gap = s["offset"].long()[:, None] - torch.arange(n, device="cuda")
    seen = (gap >= 0) & (gap < (c["window"] or 1 << 40))
    seen = seen[:, None] & chosen[:, :, 0].repeat_interleave(page, -1)
    x = torch.matmul(s["q"].float().view(B, Hkv, -1, d), gather("k").transpose(-1, -2)) / math.sqrt(d)
    if c["softcap"]:
        x = c["softcap"] * torch.tanh(x / c["softcap"])
    x.masked_fill_(~seen[:, :, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m.isinf(), 0, m))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, gather("v")) / torch.where(total == 0, 1, total)
    return o.view(B, Hq, d).to(torch.bfloat16), (m + torch.log(total)).view(B, Hq)


def _train(s):
    """O, LSE and the gradients of q, k, v, rounded to bf16 as the layers before the attention take them."""
    c = s["case"]
    B, Hq, Hkv, d, N, block = c["B"], c["Hq"], c["Hkv"], c["d"], c["Q"], c["block"]
    chosen, kinds = _choose(dict(s, bounds=_block_bounds(s["k"], block)))
    seen = chosen.repeat_interleave(block, 2)[:, :, :N].repeat_interleave(block, 3)[..., :N]
    gap = torch.arange(N, device="cuda")[:, None] - torch.arange(N, device="cuda")
    seen &= (gap >= 0) & (gap < (c["window"] or 1 << 40))
    q, do = (s[x].float().view(B, Hkv, -1, N, d) for x in ("q", "dout"))
    k, v = (s[x].float()[:, :, None] for x in ("k", "v"))
    x = torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(d)
    x.masked_fill_(~seen[:, :, None], -math.inf)
    lse = torch.logsumexp(x, -1, keepdim=True)
    p = x.sub_(torch.where(lse.isinf(), 0, lse)).exp_()
    o = torch.matmul(p, v)
    dv = torch.matmul(p.transpose(-1, -2), do).sum(2)
    ds = p * (torch.matmul(do, v.transpose(-1, -2)) - (do * o).sum(-1, keepdim=True)) / math.sqrt(d)
    dq = torch.matmul(ds, k)
    dk = torch.matmul(ds.transpose(-1, -2), q).sum(2)
    return (o.view(B, Hq, N, d).to(torch.bfloat16), lse.view(B, Hq, N), *(t.reshape(B, -1, N, d).to(torch.bfloat16) for t in (dq, dk, dv)))


# ---------------------------------------------------------------------------------------------- work
def work(case):
    c, op = case, case["op"]
    B, Hkv, d, block = c["B"], c["Hkv"], c["d"], c["block"]
    if op == "bounds":
        if c["kind"] == "dense":
            tokens, pages = B * c["N"], B * math.ceil(c["N"] / block)
        else:  # the page of the first token is read from its start: half a page on average
            new = c["N"] * (0.75 if c["ragged"] and c["N"] > 1 else 1)
            tokens, pages = B * (new + (block - 1) / 2), B * (new / block + (block - 1) / block)
        return dict(bytes=Hkv * d * (tokens * (1 if c["kind"] == "fp8" else 2) + pages * 4), flops=2 * Hkv * d * tokens)
    Hq, Q, keep = c["Hq"], c.get("Q", 1), c["keep"]
    mean = (c["lo"] + c["hi"]) / 2 if c["lo"] and B > 1 else c["hi"]
    dense = not c.get("paged", op != "train")
    bq = 1 if Q == 1 and not dense else block
    nq, nk = math.ceil(Q / bq), math.ceil(c["hi"] / block)
    reach = min(mean / block, (c["window"] or 1 << 40) / block + 1)                  # blocks that a row can see
    if dense:
        reach = min(nk / 2, reach)
    reach = max(1, reach)
    held = min(nk, mean / block) if Q > 1 else reach                               # blocks whose bounds are read, for a request and head
    choose = dict(bytes=B * Hq * Q * d * 2 + B * Hkv * (held * 4 * d + (nq * nk * 17 + 8 * nq + 8 * nk)) + B * nq * nk, flops=2 * B * Hkv * (2 * d * nq * reach + Hq // Hkv * Q * d))
    if op == "choose":
        return choose
    kept = min(keep, reach)
    if op == "train":
        pairs = B * Hq * Q * block * kept
        return dict(bytes=B * Q * d * (Hq * 8 + Hkv * 8) + B * Hq * Q * 4, flops=4 * d * pairs * 3.5)
    tokens = B * Hkv * min(kept * block, mean)
    attend = dict(bytes=tokens * 2 * (d + 4 / BLOCK if c["fp8"] else 2 * d) + B * Hq * (4 * d + 4), flops=4 * d * tokens * (Hq // Hkv))
    if op == "decode":
        return attend
    read = B * Hkv * d * (block / 2 * (1 if c["fp8"] else 2) + 4) + B * Hkv * held * 4 * d
    return dict(bytes=attend["bytes"] + read, flops=attend["flops"] + 4 * B * Hkv * d * reach)


# ---------------------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    """The definition in 64 bits, a request (and a head) at a time. A choice is whole numbers alone: nothing is given for it."""
    s = prepare(case, seed)
    c, op = case, case["op"]
    if op == "bounds" and c["kind"] == "dense":
        return torch.stack([torch.stack([torch.stack([x.double().min(1).values, x.double().max(1).values], 1) for x in k.split(c["block"], 1)], 1) for k in s["k"]])
    if op == "choose":
        return None
    bounds = _exact_pages(s) if op in ("bounds", "step") else None
    if op == "bounds":
        return bounds
    if op == "step":
        s["bounds"] = bounds
    if op == "train":
        return _exact_train(s)
    out = _exact_decode(s)
    return out if op == "decode" else (bounds, *out)


def _exact_pages(s):
    c = s["case"]
    page, out = c["block"], s["bounds"].double()
    new = s["n_new"].tolist() if "n_new" in s else [c.get("N", 1)] * c["B"]
    for b, (lo, n) in enumerate(zip(s["offset"].tolist(), new)):
        for at in range(lo - lo % page, lo + n, page) if n else ():
            pid = int(s["table"][b, at // page])
            x = s["k"][pid].double()
            if "ks" in s:
                x = (x.view(c["Hkv"], -1, BLOCK, c["d"]) * s["ks"][pid].double()[..., None, None]).view(x.shape)
            x = x[:, :lo + n - at]
            out[pid, :, 0], out[pid, :, 1] = x.min(1).values, x.max(1).values
    return out


def _exact_row(c, q, box, seen):
    """Which blocks a row keeps: queries [n, d], bounds [blocks, 2, d] and the blocks that it sees, all in 64 bits."""
    ids = seen.nonzero()[:, 0].tolist()
    if len(ids) <= c["keep"]:
        return ids
    score = torch.zeros(len(ids), dtype=torch.float64, device="cuda")
    for x in q.split(64):
        y = x[:, None, None] * box[ids][None]
        score += torch.maximum(y[:, :, 0], y[:, :, 1]).sum((0, 2))
    score = score.tolist()
    ends = set(ids[:c["first"]]) | set(ids[len(ids) - c["last"]:])
    rest = sorted((-v, j) for v, j in zip(score, ids) if j not in ends)
    return sorted(ends | {j for _, j in rest[:c["keep"] - len(ends)]})


def _exact_decode(s):
    c = s["case"]
    B, Hq, Hkv, d, page = c["B"], c["Hq"], c["Hkv"], c["d"], c["block"]
    g = Hq // Hkv
    out = torch.zeros(B, Hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")
    for b, i in enumerate(s["offset"].tolist()):
        ids = s["table"][b, :i // page + 1].long()
        j = torch.arange(len(ids) * page, device="cuda")
        hidden = (j > i) | (i - j >= (c["window"] or 1 << 40))
        seen = (~hidden).view(-1, page).any(1)
        for h in range(Hkv):
            q = s["q"][b, h * g:(h + 1) * g, 0].double()
            take = torch.tensor(_exact_row(c, q, s["bounds"][ids, h].double(), seen), device="cuda")
            k, v = (s[x][ids[take], h].double() for x in "kv")
            if c["fp8"]:
                k, v = (x.view(len(take), -1, BLOCK, d) * s[n][ids[take], h].double()[..., None, None] for x, n in ((k, "ks"), (v, "vs")))
            x = q @ k.reshape(-1, d).T * d ** -0.5
            if c["softcap"]:
                x = torch.tanh(x / c["softcap"]) * c["softcap"]
            x = x.masked_fill(hidden.view(-1, page)[take].view(1, -1), -math.inf)
            z = torch.logsumexp(x, -1)
            lse[b, h * g:(h + 1) * g] = z
            out[b, h * g:(h + 1) * g] = torch.exp(x - z[:, None]) @ v.reshape(-1, d)
    return out, lse


def _exact_train(s):
    c = s["case"]
    B, Hq, Hkv, d, N, block = c["B"], c["Hq"], c["Hkv"], c["d"], c["Q"], c["block"]
    g, nk = Hq // Hkv, (N + block - 1) // block
    q, k, v, do = (s[x].double() for x in ("q", "k", "v", "dout"))
    o, lse, dq = torch.zeros_like(q), torch.zeros(B, Hq, N, dtype=torch.float64, device="cuda"), torch.zeros_like(q)
    dk, dv = torch.zeros_like(k), torch.zeros_like(v)
    i, j = torch.arange(N, device="cuda")[:, None], torch.arange(N, device="cuda")[None]
    allowed = (j <= i) & (i - j < (c["window"] or 1 << 40))
    for b in range(B):
        for h in range(Hkv):
            box = torch.stack([torch.stack([x.min(0).values, x.max(0).values]) for x in k[b, h].split(block)])
            keep = torch.zeros(nk, nk, dtype=torch.bool, device="cuda")
            for r in range(nk):
                rows = slice(r * block, min(N, (r + 1) * block))
                seen = torch.stack([x.any() for x in allowed[rows].split(block, 1)])
                keep[r, _exact_row(c, q[b, h * g:(h + 1) * g, rows].reshape(-1, d), box, seen)] = True
            hidden = ~(allowed & keep.repeat_interleave(block, 0)[:N].repeat_interleave(block, 1)[:, :N])
            for e in range(h * g, (h + 1) * g):
                x = (q[b, e] @ k[b, h].T * d ** -0.5).masked_fill(hidden, -math.inf)
                z = torch.logsumexp(x, -1)
                p = torch.exp(x - z[:, None])
                o[b, e], lse[b, e] = p @ v[b, h], z
                dv[b, h] += p.T @ do[b, e]
                ds = p * (do[b, e] @ v[b, h].T - (do[b, e] * o[b, e]).sum(-1, keepdim=True)) * d ** -0.5
                dq[b, e] = ds @ k[b, h]
                dk[b, h] += ds.T @ q[b, e]
    return o, lse, dq, dk, dv
