"""Attention over the 8-bit paged cache on the GPU (fa_flex_decode_fp8, fa_flex_forward_paged_fp8) against 64-bit attention
over the dequantised pages: page sizes, head groups, lengths from one token, masks that leave a row empty, masked slots
that hold NaN, uneven scales, scores rules, bad pages, and a run of prompt and decode steps through the append."""
import math

import pytest
import torch

from block_sparse_masked_create_gb300 import fa
from tests import gpu_common as gc
from tests import qkv_ref as ref

pytestmark = pytest.mark.gpu
BF, F32, F8 = torch.bfloat16, torch.float32, ref.F8
NAN_BYTE = 0x7F


def gen(seed):
    return torch.Generator().manual_seed(seed)


def cache(seed, lens, Hkv, page, d, spread=1, max_pages=None, power=True):
    """Pages with N(0, 1) values (times 2^U{0..spread} a block, or any factor), scales, and the table; slots behind a
    sequence hold NaN, pages of nobody too."""
    g = gen(seed)
    each = [-(-L // page) for L in lens]
    max_pages = max_pages or max(each)
    total = sum(each) + 2
    ids = torch.randperm(total, generator=g)
    x = torch.randn(2, total, Hkv, page // 32, 32, d, generator=g)
    f = torch.exp2(torch.randint(0, spread + 1, x.shape[:4], generator=g).float())
    if not power:
        f = f * (0.5 + torch.rand(f.shape, generator=g))
    s = ref.need((x * f[..., None, None]).abs().amax((-1, -2))).float() * (1 if power else 0.7 + 0.3 * torch.rand(f.shape, generator=g))
    pages = (x * f[..., None, None] / s[..., None, None]).clamp(-448, 448).to(F8).view(2, total, Hkv, page, d)
    table = torch.full((len(lens), max_pages), -1, dtype=torch.int32)
    at = 0
    raw = pages.view(torch.uint8)
    for b, n in enumerate(each):
        table[b, :n] = ids[at:at + n].to(torch.int32)
        at += n
        if lens[b] % page:
            raw[:, table[b, n - 1], :, lens[b] % page:] = NAN_BYTE
    raw[:, ids[at:]] = NAN_BYTE
    s[:, ids[at:]] = math.nan
    return pages[0].contiguous(), pages[1].contiguous(), s[0].contiguous(), s[1].contiguous(), table


def spec_and_mask(window, prefix, i, j):
    spec = [("causal",)]
    al = j <= i
    if window:
        spec += [("window", window), ("and",)]
        al = al & (i - j < window)
    if prefix:
        spec += [("prefix", prefix), ("or",)]
        al = al | (j < prefix)
    return spec, al


def close(out, lse, want, d, softcap, dtype, extra, what):
    """O and LSE against the 64-bit result. P is rounded to fp16 (2^-11) once, 2^x and the sums are good to 2^-20; a score
    is a sum of d products in fp32, off by at most (d + 4) half steps of scale sum |q k|, and by 2^-21 of a soft-cap
    (1 - 2 / (1 + e^2u): rcp and 2^x good to 2^-22 each)."""
    o, z, av, qk = want
    ds = ((d + 4) * ref.U32 * qk + softcap * 2.0 ** -21 + extra)[..., None]
    bound = (2.0 ** -11 + 2.0 ** -20 + 2 * ds) * av
    bound = bound + ref.HALF[dtype] * (o.abs() + bound)
    err = (out.double().cpu() - o).abs()
    assert torch.isfinite(out.float()).all(), what
    assert (err <= bound).all(), f"{what}: O {float((err - bound).max()):.3e} over the bound"
    empty = z.isinf()
    assert torch.equal(lse.cpu().isneginf(), empty), what
    lerr = (lse.double().cpu() - z).abs()[~empty]
    lb = (ds[..., 0] + 2.0 ** -20 + 4 * ref.U32 * z.abs())[~empty]
    assert (lerr <= lb).all(), f"{what}: LSE {float((lerr - lb).max()):.3e} over the bound"


def run_decode(seed, lens, Hq, Hkv, d, page, window=0, prefix=0, softcap=0.0, alibi=False, rel=False, dtype=F32, spread=1,
               max_pages=None, power=True, offset=None, q_scale=1.0):
    kp, vp, ks, vs, table = cache(seed, lens, Hkv, page, d, spread, max_pages, power)
    g = gen(seed + 1)
    B = len(lens)
    q = (torch.randn(B, Hq, d, generator=g) * q_scale).to(BF)
    off = torch.tensor([L - 1 for L in lens] if offset is None else offset, dtype=torch.int32)
    n = table.shape[1] * page
    slopes = 2.0 ** (-8.0 * torch.arange(1, Hq + 1) / Hq) if alibi else None
    table_rel = torch.randn(Hq, 2 * n - 1, generator=g) if rel else None
    off_c = off.cuda()
    spec, _ = spec_and_mask(window, prefix, torch.zeros(1, 1), torch.zeros(1, 1))
    bm = fa.create_block_mask(fa.make_mask_rule(spec, q_offset=off_c, batch_dependent=True), B, Hq, 1, n, 1, page, keep=[off_c])
    sc = fa.make_score_rule(None if slopes is None else slopes.cuda(), None if table_rel is None else table_rel.cuda(), softcap)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = [t.cuda() for t in (q, kp, vp, ks, vs, table)]
    out, lse = fa.flex_decode_fp8(*args, bm, sc, status=status, out_dtype=dtype)
    st = fa.check_status(status)
    dk, dv = ref.dequant(kp, ks), ref.dequant(vp, vs)
    for b in range(B):
        i, j = torch.tensor([[int(off[b])]]), torch.arange(lens[b])[None]
        _, al = spec_and_mask(window, prefix, i, j)
        want = ref.attention(q[b, :, None].double(), ref.gather(dk, table[b], lens[b]), ref.gather(dv, table[b], lens[b]), al,
                             d ** -0.5, slopes, i[:, 0], softcap, table_rel, n)
        extra = 4 * ref.U32 * (max(lens) if alibi else 8)  # ALiBi's product with a distance, the bias's sum
        close(out[b][:, None], lse[b][:, None], want, d, softcap, dtype, extra, f"request {b} of {lens}")
    return out, lse, st, args, bm, sc


@pytest.mark.parametrize("page", [32, 64, 128])
@pytest.mark.parametrize("g,d", [(1, 64), (3, 128), (4, 128), (8, 64), (9, 128), (16, 64)])
def test_decode_groups_and_pages(page, g, d):
    _, _, st, _, _, _ = run_decode(1, [1, 31, 32, 33, page, 5 * page + 7, 701], 2 * g, 2, d, page)
    assert st == fa.OK


@pytest.mark.parametrize("kw", [dict(window=40), dict(window=1), dict(prefix=45), dict(softcap=20.0), dict(alibi=True), dict(rel=True),
                                dict(window=300, softcap=15.0, alibi=True), dict(dtype=BF), dict(spread=30, power=False),
                                dict(q_scale=1e-12), dict(q_scale=30.0), dict(dtype=BF, power=False)], ids=str)
def test_decode_rules_types_and_scales(kw):
    lens = [77, 1000, 2050, 64]
    _, _, st, _, _, _ = run_decode(3, lens, 8, 2, 128, 64, **kw)
    assert st == fa.OK


def test_decode_spans_and_long_table():
    # a table far longer than the sequences: spans of 4096 tokens, one of them the whole of a short request
    _, _, st, _, _, _ = run_decode(5, [9000, 100, 4096, 4097, 1], 4, 1, 64, 64, max_pages=4000)
    assert st == fa.OK


@pytest.mark.parametrize("kw", [dict(window=1), dict(window=64), dict(window=65), dict(window=700), dict(prefix=64), dict(prefix=65, window=129),
                                dict(window=10 ** 9)], ids=str)
def test_decode_bounded_rules_over_a_long_table(kw):
    # the spans are cut for what the rule can see, which starts anywhere in a page (a prefix is a part of every sequence:
    # the rule shows its keys to all rows)
    short = max(1, kw.get("prefix", 1))
    for shift in (0, 1, 63):
        _, _, st, _, _, _ = run_decode(14 + shift, [3000 + shift, short + 64 + shift, short], 4, 1, 64, 64, max_pages=900, **kw)
        assert st == fa.OK


def test_decode_empty_rows():
    out, lse, st, _, _, _ = run_decode(6, [50, 50], 4, 2, 64, 32, offset=[-1, 49])
    assert st == fa.OK and not out[0].any() and lse[0].isneginf().all()


def test_decode_documents():
    page, d, H, L = 32, 64, 2, 300
    kp, vp, ks, vs, table = cache(8, [L], H, page, d)
    n = table.shape[1] * page
    ids = (torch.arange(n) // 50 % 3).to(torch.int32)[None]  # unsorted
    q = torch.randn(1, H, d, generator=gen(9)).to(BF)
    off = torch.tensor([L - 1], dtype=torch.int32).cuda()
    doc = ids.cuda()
    rule = fa.make_mask_rule([("causal",), ("doc",), ("and",)], doc_ids=doc, q_offset=off)
    bm = fa.create_block_mask(rule, 1, H, 1, n, 1, page, keep=[doc, off])
    out, lse = fa.flex_decode_fp8(*[t.cuda() for t in (q, kp, vp, ks, vs, table)], bm, out_dtype=F32)
    al = (ids[0, :L] == ids[0, L - 1])[None]
    want = ref.attention(q[0][:, None].double(), ref.gather(ref.dequant(kp, ks), table[0], L), ref.gather(ref.dequant(vp, vs), table[0], L),
                         al, d ** -0.5, pos=torch.tensor([L - 1]))
    close(out[0][:, None], lse[0][:, None], want, d, 0.0, F32, 0.0, "documents")


def test_decode_bad_page_is_reported_and_skipped():
    kp, vp, ks, vs, table = cache(10, [100, 200], 2, 32, 64)
    table[0, 1], table[1, 3] = 10 ** 6, -7
    off = torch.tensor([99, 199], dtype=torch.int32).cuda()
    bm = fa.create_block_mask(fa.make_mask_rule([("causal",)], q_offset=off), 2, 4, 1, table.shape[1] * 32, 1, 32, keep=[off])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = torch.randn(2, 4, 64, generator=gen(11)).to(BF)
    out, _ = fa.flex_decode_fp8(*[t.cuda() for t in (q, kp, vp, ks, vs, table)], bm, status=status)
    assert fa.check_status(status) == fa.ERR_DEVICE_CHECK and torch.isfinite(out.float()).all()


def test_decode_two_streams_two_graphs_and_counters():
    out, lse, _, args, bm, sc = run_decode(12, [700, 1500], 8, 2, 128, 64)
    need = fa.decode_fp8_workspace_bytes(2, 8, 2, 128, args[5].shape[1], 64)
    runs = []
    for i in range(2):  # each with a workspace of its own, replayed against each other
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        o, l = torch.empty_like(out), torch.empty_like(lse)
        with torch.cuda.stream(s):
            fa.flex_decode_fp8(*args, bm, sc, out=o, lse=l, workspace=ws)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                fa.flex_decode_fp8(*args, bm, sc, out=o, lse=l, workspace=ws)
        runs.append((s, graph, o, l, ws))
    torch.cuda.synchronize()
    for _, _, o, l, _ in runs:
        o.fill_(math.nan)
        l.fill_(math.nan)
    torch.cuda.synchronize()
    for _ in range(5):
        for s, graph, _, _, _ in runs:
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for _, _, o, l, _ in runs:
        assert torch.equal(o, out) and torch.equal(l, lse)
    cnt = torch.zeros(4, dtype=torch.int64, device="cuda")
    fa.flex_decode_fp8(*args, bm, sc, counters=cnt)
    assert int(cnt[3]) == 2 * 2 * sum(-(-L // 64) for L in (700, 1500))


# ------------------------------------------------------------------------------------------ chunks of queries
def prefill_case(seed, lens, Q, Hq, Hkv, d, page, window=0, prefix=0, bk=128, power=True):
    kp, vp, ks, vs, table = cache(seed, lens, Hkv, page, d, power=power)
    B, kv_len = len(lens), max(lens)
    q = torch.randn(B, Hq, Q, d, generator=gen(seed + 1)).to(BF)
    off = torch.tensor([L - Q for L in lens], dtype=torch.int32).cuda()
    spec, _ = spec_and_mask(window, prefix, torch.zeros(1, 1), torch.zeros(1, 1))
    bm = fa.create_block_mask(fa.make_mask_rule(spec, q_offset=off), B, Hq, Q, kv_len, bk, bk, keep=[off])
    return q, kp, vp, ks, vs, table, bm, off, kv_len


@pytest.mark.parametrize("page,bk,Q,Hq,Hkv,d,window,softcap,alibi", [
    (128, 128, 100, 4, 2, 128, 0, 0.0, False), (32, 128, 1, 2, 2, 64, 0, 0.0, False), (64, 128, 129, 4, 1, 128, 150, 20.0, False),
    (128, 64, 70, 4, 4, 64, 0, 0.0, True), (64, 32, 33, 2, 1, 128, 40, 0.0, False), (32, 64, 300, 3, 1, 64, 0, 0.0, False), (64, 128, 150, 16, 1, 64, 0, 0.0, True),
    (128, 128, 700, 3, 1, 128, 200, 0.0, False)])
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_prefill_matches_64_bits_and_the_bf16_forward(page, bk, Q, Hq, Hkv, d, window, softcap, alibi, dtype):
    lens = [Q, Q + 1, Q + 333]
    q, kp, vp, ks, vs, table, bm, off, kv_len = prefill_case(20, lens, Q, Hq, Hkv, d, page, window, bk=bk)
    slopes = 2.0 ** (-8.0 * torch.arange(1, Hq + 1) / Hq) if alibi else None
    sc = fa.make_score_rule(None if slopes is None else slopes.cuda(), None, softcap)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = [t.cuda() for t in (q, kp, vp, ks, vs, table)]
    out, lse = fa.flex_forward_paged_fp8(*args, bm, kv_len, sc, status=status, out_dtype=dtype, chunk_blocks=-1)
    assert fa.check_status(status) == fa.OK
    dk, dv = ref.dequant(kp, ks), ref.dequant(vp, vs)
    expanded = bk != 128 or -(-Q // 128) * (Hq // Hkv) > 16  # many query tiles to a key block
    if expanded:
        # power-of-two scales: the expanded values are the cached ones, so the bf16 forward over them gives the same bits
        k, v = (torch.stack([torch.cat([ref.gather(t, table[b], L), torch.zeros(Hkv, kv_len - L, d, dtype=torch.float64)], 1)
                             for b, L in enumerate(lens)]).to(BF).cuda() for t in (dk, dv))
        o2, l2 = fa.flex_forward(args[0], k, v, bm, sc, out_dtype=dtype)
        assert torch.equal(out, o2) and torch.equal(lse, l2)
    for b, L in enumerate(lens):
        i, j = L - Q + torch.arange(Q)[:, None], torch.arange(L)[None]
        _, al = spec_and_mask(window, 0, i, j)
        want = ref.attention(q[b].double(), ref.gather(dk, table[b], L), ref.gather(dv, table[b], L), al, d ** -0.5, slopes, i[:, 0], softcap)
        # ALiBi: the bias is stepped by 8 columns, at most 16 roundings of its size a block, and a product with a distance
        extra = 20 * ref.U32 * L if alibi else 0.0
        if not expanded:
            close(out[b], lse[b], want, d, softcap, dtype, extra, f"request {b}")
        else:
            # the cached values are N(0, 1) times 1 or 2: the forward's tolerance for N(0, 1), doubled
            gc.compare(out[b].float().cpu().numpy() / 2, lse[b].cpu().numpy(), want[0].numpy() / 2, want[1].numpy(), "prefill",
                       out_bf16=dtype == BF)


@pytest.mark.parametrize("kw", [dict(prefix=70), dict(window=1), dict(softcap=100.0), dict(rel=True), dict(alibi=True, softcap=30.0), dict(doc=True),
                                dict(spread=9), dict(power=False), dict(q_scale=1e-20), dict(dense=True)], ids=str)
@pytest.mark.parametrize("d,page,Q", [(128, 64, 150), (64, 128, 150), (128, 128, 30), (64, 32, 1)])
def test_prefill_rules_and_scales(kw, d, page, Q):
    # 128 x 128 blocks: every score path, document masks, V scales up to 2^9 apart in a block, a rule without a causal bound;
    # few queries: the heads of a KV head share a tile
    Hq, Hkv, lens = (4, 2, [150, 390]) if Q == 150 else (6, 2, [150, 390])
    kp, vp, ks, vs, table = cache(40, lens, Hkv, page, d, kw.get("spread", 1), power=kw.get("power", True))
    B, n = len(lens), max(lens)
    if kw.get("dense"):
        lens = [n, n]
        kp, vp, ks, vs, table = cache(40, lens, Hkv, page, d)
    g = gen(41)
    q = (torch.randn(B, Hq, Q, d, generator=g) * kw.get("q_scale", 1.0)).to(BF)
    off = torch.tensor([L - Q for L in lens], dtype=torch.int32).cuda()
    slopes = 2.0 ** (-8.0 * torch.arange(1, Hq + 1) / Hq) if kw.get("alibi") else None
    rel = torch.randn(Hq, 2 * n - 1, generator=g) if kw.get("rel") else None
    spec, _ = spec_and_mask(kw.get("window", 0), kw.get("prefix", 0), torch.zeros(1, 1), torch.zeros(1, 1))
    doc = (torch.arange(n) // 60 % 4).to(torch.int32)[None] if kw.get("doc") else None
    if kw.get("doc"):
        spec += [("doc",), ("and",)]
    if kw.get("dense"):
        spec = [("true",)]
    doc_c = None if doc is None else doc.cuda()
    bm = fa.create_block_mask(fa.make_mask_rule(spec, doc_ids=doc_c, q_offset=off), B, Hq, Q, n, 128, 128, keep=[off, doc_c])
    cap = kw.get("softcap", 0.0)
    sc = fa.make_score_rule(None if slopes is None else slopes.cuda(), None if rel is None else rel.cuda(), cap)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = [t.cuda() for t in (q, kp, vp, ks, vs, table)]
    out, lse = fa.flex_forward_paged_fp8(*args, bm, n, sc, status=status, out_dtype=F32)
    cut, cut_lse = fa.flex_forward_paged_fp8(*args, bm, n, sc, status=status, out_dtype=F32, chunk_blocks=1)
    assert fa.check_status(status) == fa.OK
    dk, dv = ref.dequant(kp, ks), ref.dequant(vp, vs)
    for b, L in enumerate(lens):
        i, j = L - Q + torch.arange(Q)[:, None], torch.arange(L)[None]
        _, al = spec_and_mask(kw.get("window", 0), kw.get("prefix", 0), i, j)
        if doc is not None:
            al = al & (doc[0, :L][None] == doc[0, i[:, 0]][:, None])
        if kw.get("dense"):
            al = torch.ones_like(al)
        want = ref.attention(q[b].double(), ref.gather(dk, table[b], L), ref.gather(dv, table[b], L), al, d ** -0.5, slopes, i[:, 0], cap, rel, n)
        # P in fp16 relative to a block's largest V scale: 2^-25 of 448 such scales for a key whose P is subnormal there
        floor = 2.0 ** -25 * 448 * float(vs[table[b, :-(-L // page)].long()].nan_to_num(0).max()) * L if kw.get("spread") else 0.0
        want = (want[0], want[1], want[2] + floor * 2.0 ** 11, want[3])
        close(out[b], lse[b], want, d, cap, F32, 20 * ref.U32 * (L + 8), f"request {b} {kw}")
        # cut into single key blocks and merged in fp32: 4 more roundings of the sums, and 2^x of differences of LSEs
        close(cut[b], cut_lse[b], want, d, cap, F32, 20 * ref.U32 * (L + 8) + 2.0 ** -18, f"cut, request {b} {kw}")


def test_prefill_cut_rows():
    # few rows over a long context: the library cuts them by itself; the result is the uncut one up to the order of sums
    lens = [6000, 5000]
    q, kp, vp, ks, vs, table, bm, off, kv_len = prefill_case(22, lens, 40, 4, 2, 128, 64)
    args = [t.cuda() for t in (q, kp, vp, ks, vs, table)]
    whole = fa.flex_forward_paged_fp8(*args, bm, kv_len, chunk_blocks=-1, out_dtype=F32)
    assert fa.forward_paged_fp8_workspace_bytes(bm, 2, 4, 2, 128, 0) > fa.forward_paged_fp8_workspace_bytes(bm, 2, 4, 2, 128, -1)
    for chunk in (0, 1, 7):  # (cut rows over expanded blocks: below)
        o, l = fa.flex_forward_paged_fp8(*args, bm, kv_len, chunk_blocks=chunk, out_dtype=F32)
        # each side has its own rounding of P to fp16 (2^-11 of a weighted mean of |v| below 2), and the merge's fp32
        assert (o - whole[0]).abs().max() <= 2 * 2.0 ** -11 * 2 + 1e-5 and (l - whole[1]).abs().max() <= 2e-5


def test_prefill_cut_rows_over_expanded_blocks():
    lens = [1500]
    q, kp, vp, ks, vs, table, bm, off, kv_len = prefill_case(23, lens, 400, 8, 1, 64, 128)  # 32 query tiles to a key block
    args = [t.cuda() for t in (q, kp, vp, ks, vs, table)]
    whole = fa.flex_forward_paged_fp8(*args, bm, kv_len, chunk_blocks=-1, out_dtype=F32)
    o, l = fa.flex_forward_paged_fp8(*args, bm, kv_len, chunk_blocks=3, out_dtype=F32)
    # each side has its own rounding of P to bf16 (2^-8 of a weighted mean of |v| below 2)
    assert (o - whole[0]).abs().max() <= 2 * 2.0 ** -8 * 2 and (l - whole[1]).abs().max() <= 2e-3


def test_prefill_scales_that_are_no_powers_of_two_in_small_blocks():
    lens, Q = [200, 260], 130
    q, kp, vp, ks, vs, table, bm, off, kv_len = prefill_case(24, lens, Q, 2, 2, 64, 32, bk=64, power=False)
    out, lse = fa.flex_forward_paged_fp8(*[t.cuda() for t in (q, kp, vp, ks, vs, table)], bm, kv_len, out_dtype=F32)
    dk, dv = (ref.dequant(p, s).float().to(BF).double() for p, s in ((kp, ks), (vp, vs)))  # the values rounded to bf16
    for b, L in enumerate(lens):
        i, j = L - Q + torch.arange(Q)[:, None], torch.arange(L)[None]
        o, z, av, qk = ref.attention(q[b].double(), ref.gather(dk, table[b], L), ref.gather(dv, table[b], L), j <= i, 0.125, pos=i[:, 0])
        # fp32 products and P in bf16
        assert ((out[b].double().cpu() - o).abs() <= (2.0 ** -8 + 2.0 ** -10) * av + 1e-4).all()
        assert (lse[b].double().cpu() - z).abs().max() <= 2e-3


def test_prefill_bad_page_is_reported():
    q, kp, vp, ks, vs, table, bm, off, kv_len = prefill_case(26, [300], 20, 2, 2, 64, 64)
    table[0, 2] = 12345
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, _ = fa.flex_forward_paged_fp8(*[t.cuda() for t in (q, kp, vp, ks, vs, table)], bm, kv_len, status=status)
    assert fa.check_status(status) == fa.ERR_DEVICE_CHECK and torch.isfinite(out.float()).all()


# ------------------------------------------------------------------------------------------ a serving run
@pytest.mark.parametrize("fp8", [True, False])
def test_prompt_then_decode_steps(fp8):
    """A padded batch of prompts into the cache, attention over the chunk, then single tokens appended and decoded; each
    step against 64-bit attention over what the cache then holds."""
    B, Q, Hq, Hkv, d, page, steps = 3, 90, 8, 2, 64, 64, 4
    g = gen(30)
    lens = [90, 41, 64]
    each = -(-(Q + steps) // page)
    table = torch.randperm(B * each + 1, generator=g)[:B * each].view(B, each).to(torch.int32)
    f = (10000.0 ** (-2 * torch.arange(d // 2, dtype=torch.float64) / d)).float().cuda()
    w = [(1 + 0.2 * torch.randn(d, generator=g)).cuda() for _ in range(2)]
    rule = fa.make_qk_rule(*w, 1e-6, f)
    kp, vp = (torch.full((B * each + 1, Hkv, page, d), NAN_BYTE, dtype=torch.uint8, device="cuda").view(F8) if fp8 else
              torch.zeros(B * each + 1, Hkv, page, d, dtype=BF, device="cuda") for _ in range(2))
    sc = [torch.full((B * each + 1, Hkv, page // 32), math.nan, device="cuda") for _ in range(2)] if fp8 else []
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    n_new = torch.tensor(lens, dtype=torch.int32).cuda()
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    t_c = table.cuda()
    append = fa.kv_append_fp8 if fp8 else fa.kv_append

    def rows(n):
        return torch.randn(B, n, Hq + 2 * Hkv, d, generator=g).to(BF).cuda().split([Hq, Hkv, Hkv], dim=2)

    def held():
        return [ref.dequant(p.cpu(), s.cpu()) for p, s in ((kp, sc[0]), (vp, sc[1]))] if fp8 else [p.cpu().double() for p in (kp, vp)]

    q = append(*rows(Q), kp, vp, *sc, t_c, rule, zero, n_new, torch.zeros(B, Hq, Q, d, dtype=BF, device="cuda"), status)
    assert fa.check_status(status) == fa.OK
    if fp8:  # rows behind a shorter prompt see keys that nobody appended; only the prompt's own rows are looked at
        bm = fa.create_block_mask(fa.make_mask_rule([("causal",)]), B, Hq, Q, Q, 128, 128)
        kd, vd = held()
        for b, L in enumerate(lens):
            one = fa.create_block_mask(fa.make_mask_rule([("causal",)]), 1, Hq, L, L, 128, 128)
            o, l = fa.flex_forward_paged_fp8(q[b:b + 1, :, :L].contiguous(), kp, vp, *sc, t_c[b:b + 1].contiguous(), one, L, status=status,
                                             out_dtype=F32)
            i, j = torch.arange(L)[:, None], torch.arange(L)[None]
            want, z, av, _ = ref.attention(q[b, :, :L].double().cpu(), ref.gather(kd, table[b], L), ref.gather(vd, table[b], L), j <= i, 0.125,
                                           pos=i[:, 0])
            assert ((o[0].double().cpu() - want).abs() <= (2.0 ** -8 + 2.0 ** -10) * av + 1e-4).all()
            assert (l[0].double().cpu() - z).abs().max() <= 2e-3
        assert fa.check_status(status) == fa.OK and bm.shape[0] == 1
    for step in range(steps):
        pos = (n_new + step).contiguous()
        q = append(*rows(1), kp, vp, *sc, t_c, rule, pos, status=status)
        bm = fa.create_block_mask(fa.make_mask_rule([("causal",)], q_offset=pos), B, Hq, 1, each * page, 1, page, keep=[pos])
        decode = fa.flex_decode_fp8 if fp8 else fa.flex_decode
        o, l = decode(q[:, :, 0], kp, vp, *sc, t_c, bm, status=status, out_dtype=F32)
        assert fa.check_status(status) == fa.OK
        kd, vd = held()
        for b, L in enumerate(lens):
            n = L + step + 1
            want = ref.attention(q[b].double().cpu(), ref.gather(kd, table[b], n), ref.gather(vd, table[b], n), torch.ones(1, n, dtype=torch.bool),
                                 0.125, pos=torch.tensor([n - 1]))
            if fp8:
                close(o[b][:, None], l[b][:, None], want, d, 0.0, F32, 0.0, f"step {step} request {b}")
            else:
                assert ((o[b][:, None].double().cpu() - want[0]).abs() <= 2.0 ** -7 * want[2] + 1e-4).all()


def test_pool_past_32_bit_offsets():
    # pages that lie behind 4 GiB of a pool: append, decode and prefill give what they give in a small pool
    Hq, Hkv, d, page, far = 8, 8, 128, 128, 2 ** 32 // (8 * 128 * 128)
    g = gen(50)
    x = torch.randn(1, 300, Hq + 2 * Hkv, d, generator=g).to(BF).cuda()
    q, k, v = x.split([Hq, Hkv, Hkv], dim=2)
    f = (10000.0 ** (-2 * torch.arange(d // 2, dtype=torch.float64) / d)).float().cuda()
    rule = fa.make_qk_rule(None, None, 1e-6, f)
    off = torch.tensor([299], dtype=torch.int32).cuda()
    mask = fa.create_block_mask(fa.make_mask_rule([("causal",)], q_offset=off), 1, Hq, 1, 3 * page, 1, page, keep=[off])
    chunk = fa.create_block_mask(fa.make_mask_rule([("causal",)]), 1, Hq, 299, 299, 128, 128)
    small = fa.create_block_mask(fa.make_mask_rule([("causal",)]), 1, Hq, 299, 299, 64, 64)
    got = []
    for first in (0, far):
        kp, vp = (torch.zeros(first + 3, Hkv, page, d, dtype=torch.uint8, device="cuda").view(F8) for _ in range(2))
        ks, vs = (torch.zeros(first + 3, Hkv, page // 32, device="cuda") for _ in range(2))
        table = torch.tensor([[first + 2, first, first + 1]], dtype=torch.int32).cuda()
        cache_ = (kp, vp, ks, vs, table)
        qp = fa.kv_append_fp8(q[:, :299], k[:, :299], v[:, :299], *cache_, rule)
        qd = fa.kv_append_fp8(q[:, 299:], k[:, 299:], v[:, 299:], *cache_, rule, off)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got.append((*fa.flex_decode_fp8(qd[:, :, 0], *cache_, mask, status=status), *fa.flex_forward_paged_fp8(qp, *cache_, chunk, 299, status=status),
                    *fa.flex_forward_paged_fp8(qp, *cache_, small, 299, status=status), kp[first:].view(torch.uint8).clone(), ks[first:].clone()))
        assert fa.check_status(status) == fa.OK and kp[first:].float().any()
    for a, b in zip(*got):
        assert torch.equal(a, b)
