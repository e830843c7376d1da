"""Bounds of key blocks, blocks chosen by them, and attention over the chosen blocks, against plain 64-bit forms."""
import math

import numpy as np
import pytest
import torch

import select_ref as ref
from gpu_common import LSE_MAX, O_MAX, O_MEAN, tables_np

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module")
def fa():
    from block_sparse_masked_create_gb300 import fa as m
    m.load()
    return m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def bf(shape, seed, spread=True):
    g = gen(seed)
    x = torch.randn(shape, generator=g, device="cuda")
    if spread:
        x *= 1 + 7 * (torch.rand(shape[-1], generator=g, device="cuda") > 0.9)
    return x.to(BF)


def same_bounds(got, want):
    got, want = got.double().cpu(), want.double()
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.nan_to_num(0.0), want.nan_to_num(0.0))


# ---------------------------------------------------------------------------------------------- bounds
@pytest.mark.parametrize("B,H,N,d,Bk", [(1, 1, 1, 64, 128), (2, 3, 1000, 128, 128), (1, 2, 257, 64, 64), (3, 1, 129, 128, 1), (1, 2, 77, 64, 33),
                                        (2, 2, 640, 128, 16), (1, 1, 5, 128, 127), (1, 1, 40000, 64, 32)])
def test_key_bounds(fa, B, H, N, d, Bk):
    k = bf((B, H, N, d), N + Bk)
    same_bounds(fa.key_bounds(k, Bk), ref.key_bounds(k, Bk))


def test_key_bounds_of_infinities_nan_and_zeros(fa):
    k = bf((1, 2, 300, 64), 3)
    k[0, 0, 5, 3], k[0, 0, 6, 3], k[0, 0, 150, 7], k[0, 1, 299, 63], k[0, 1, 128:256, 2] = math.inf, -math.inf, math.nan, math.nan, -0.0
    k[0, 1, 0:128] = torch.finfo(BF).min
    same_bounds(fa.key_bounds(k, 128), ref.key_bounds(k, 128))


def cache(P, H, page, d, seed, fp8, odd_scales=False):
    x = bf((P, H, page, d), seed)
    if not fp8:
        return x, None
    g = gen(seed + 1)
    s = torch.exp2(torch.randint(-6, 3, (P, H, page // 32), generator=g, device="cuda").float())
    if odd_scales:
        s *= 1 + torch.rand(s.shape, generator=g, device="cuda")
    return x.to(ref.F8), s


def values(pages, scale, dtype=torch.float64):
    if scale is None:
        return pages.to(dtype)
    P, H, page, d = pages.shape
    return (pages.to(dtype).view(P, H, page // 32, 32, d) * scale.to(dtype)[..., None, None]).view(P, H, page, d)


@pytest.mark.parametrize("fp8,page,d", [(False, 16, 64), (False, 64, 128), (False, 128, 64), (True, 32, 128), (True, 64, 64), (True, 128, 128)])
@pytest.mark.parametrize("N", [1, 5, 300])
def test_page_bounds(fa, fp8, page, d, N):
    B, H, width = 5, 3, (300 + N) // page + 2
    P = B * width + 2
    pages, scale = cache(P, H, page, d, page + N, fp8)
    table = torch.randperm(P, generator=gen(1), device="cuda")[:B * width].to(torch.int32).view(B, width)
    off = torch.tensor([0, page - 1, page, 299, 31], dtype=torch.int32, device="cuda")
    n_new = torch.tensor([N, N, 0, max(1, N // 2), N], dtype=torch.int32, device="cuda")
    was = torch.full((P, H, 2, d), 7.0, dtype=BF, device="cuda")
    want = was.double().cpu()
    x = values(pages, scale).cpu()
    raw = pages.view(torch.uint8) if fp8 else pages
    for b in range(B):
        lo, hi = int(off[b]), int(off[b] + n_new[b])
        for t in range(width):
            pid, held = int(table[b, t]), min(page, hi - t * page)
            if held < page:
                raw[pid, :, max(held, 0):] = 0x7F if fp8 else math.nan      # slots that nobody wrote
            if n_new[b] and lo // page <= t <= (hi - 1) // page:
                want[pid] = torch.stack([x[pid, :, :held].amin(1), x[pid, :, :held].amax(1)], 1)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (table, N, off, n_new, status)
    got = fa.kv_bounds_fp8(pages, scale, was, *args) if fp8 else fa.kv_bounds(pages, was, *args)
    assert got is was
    assert fa.check_status(status) == fa.OK
    same_bounds(got, want)


def test_page_bounds_round_outwards(fa):
    pages, scale = cache(9, 2, 64, 128, 5, True, odd_scales=True)
    scale[3, 0, 0], scale[4, 1, 1], scale[5, 0, 1] = math.nan, math.inf, 0.0      # read as 2^-40, 2^40 and 2^-40
    pages.view(torch.uint8)[6, 1, 10, 5] = 0x7F
    table = torch.arange(9, dtype=torch.int32, device="cuda").view(1, 9)
    got = fa.kv_bounds_fp8(pages, scale, torch.zeros(9, 2, 2, 128, dtype=BF, device="cuda"), table, 9 * 64).double()
    x = values(pages, torch.where(scale.isnan(), torch.zeros_like(scale), scale).clamp(2.0**-40, 2.0**40))
    lo, hi = x.amin(2), x.amax(2)
    assert torch.equal(got.isnan(), torch.stack([lo, hi], 2).isnan()) and bool(got[6, 1, 0, 5].isnan())
    lo, hi, a, b = (t.nan_to_num(0.0) for t in (lo, hi, got[:, :, 0], got[:, :, 1]))
    assert bool((a <= lo).all() and (b >= hi).all())
    # one bf16 step outwards, 2^-7 of the value at most, and the fp32 product's step
    assert bool(((lo - a) <= lo.abs() * (2.0**-7 + 2.0**-22)).all() and ((b - hi) <= hi.abs() * (2.0**-7 + 2.0**-22)).all())


def test_page_bounds_out_of_range(fa):
    pages, _ = cache(8, 2, 32, 64, 9, False)
    table = torch.tensor([[0, 1, 2], [3, 99, 4], [5, 6, -1], [7, 7, 7]], dtype=torch.int32, device="cuda")
    zero = torch.zeros(8, 2, 2, 64, dtype=BF, device="cuda")

    def run(off, n, N):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        t = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        out = fa.kv_bounds(pages, zero.clone(), table, N, t(off), t(n), status)
        return fa.check_status(status), out.double().cpu()

    x = pages.double().cpu()
    box = lambda p, n: torch.stack([x[p, :, :n].amin(1), x[p, :, :n].amax(1)], 1)  # noqa: E731
    st, out = run([90, 0, 0, 0], [10, 1, 1, 0], 10)      # request 0 runs past its 96 slots: those that fit count
    assert st == fa.ERR_DEVICE_CHECK
    same_bounds(out[2], box(2, 32))
    same_bounds(out[3], box(3, 1))
    assert not out[[0, 1, 4, 6, 7]].any()
    st, out = run([-5, 20, 0, 0], [10, 30, 30, 0], 30)   # before the start; a page id past the pool
    assert st == fa.ERR_DEVICE_CHECK
    same_bounds(out[0], box(0, 5))
    same_bounds(out[3], box(3, 32))
    assert not out[[1, 2, 4]].any()
    st, out = run([0, 0, 0, 0], [0, 0, 31, -1], 30)      # counts outside 0 .. N are clamped
    assert st == fa.ERR_DEVICE_CHECK
    same_bounds(out[5], box(5, 30))
    st, out = run([2**31 - 1, 0, 0, 0], [5, 0, 0, 0], 5)
    assert st == fa.ERR_DEVICE_CHECK and not out.any()
    assert run([0, 0, 0, 0], [0, 0, 0, 0], 30)[0] == fa.OK


def test_page_bounds_of_few_where_many_may_be_new(fa):
    pages, _ = cache(6, 2, 16, 64, 12, False)
    table = torch.tensor([[0, 1, 2], [5, 4, 3]], dtype=torch.int32, device="cuda")
    t = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = fa.kv_bounds(pages, torch.zeros(6, 2, 2, 64, dtype=BF, device="cuda"), table, 2**31 - 1, t([40, 10]), t([8, 20]), status)
    assert fa.check_status(status) == fa.OK
    want = torch.zeros(6, 2, 2, 64, dtype=torch.float64)
    for p, n in ((2, 16), (5, 16), (4, 14)):
        x = pages[p, :, :n].double().cpu()
        want[p] = torch.stack([x.amin(1), x.amax(1)], 1)
    same_bounds(out, want)


# ---------------------------------------------------------------------------------------------- the choice
MANY = 700  # queries in blocks of one: rows enough for CTAs that take several


def block_of(Q):
    return 1 if Q == MANY else 128


def same_tables(bm, cls):
    got, want = tables_np(bm), ref.tables(cls)
    assert set(got) == set(want)
    for name in want:
        assert got[name].shape == want[name].shape and np.array_equal(got[name], want[name]), name


def boxes(shape, seed):
    """Bounds [..., 2, d] about centres of their own."""
    g = gen(seed)
    c = torch.randn(*shape[:-2], 1, shape[-1], generator=g, device="cuda")
    h = 1 + torch.rand(shape, generator=g, device="cuda")
    h[..., 0, :] *= -1
    return ((c + h) * (1 + 7 * (torch.rand(shape[-1], generator=g, device="cuda") > 0.9))).to(BF)


def paged_case(fa, B, lens, Hq, Hkv, d, page, seed, spec=(("causal",),), Q=1, bq=1, P_extra=3):
    width = (max(lens) + page - 1) // page
    P = B * width + P_extra
    table = torch.randperm(P, generator=gen(seed), device="cuda")[:B * width].to(torch.int32).view(B, width)
    for b, n in enumerate(lens):
        table[b, (n + page - 1) // page:] = -1
    off = torch.tensor([n - Q for n in lens], dtype=torch.int32, device="cuda")
    rule = fa.make_mask_rule(list(spec), q_offset=off)
    src = fa.create_block_mask(rule, B, Hq, Q, width * page, bq, page)
    q = bf((B, Hq, Q, d), seed + 1, spread=False)
    return src, q, boxes((P, Hkv, 2, d), seed + 2), table, off


@pytest.mark.parametrize("B,lens,Hq,Hkv,d,page,keep,first,last,spec", [
    (1, [1], 1, 1, 64, 32, 1, 0, 1, [("causal",)]),                                        # one block
    (3, [600, 33, 257], 4, 2, 64, 32, 8, 1, 2, [("causal",)]),                             # one row short of a choice
    (2, [4000, 2100], 32, 8, 128, 64, 5, 0, 0, [("causal",)]),                             # nothing is kept always
    (5, [999, 1, 64, 65, 128], 6, 2, 128, 64, 3, 1, 2, [("causal",)]),                     # the ends alone
    (2, [3000, 2500], 8, 8, 64, 128, 4, 1, 1, [("causal",), ("window", 1500), ("and",)]),
    (2, [3000, 2500], 16, 1, 128, 32, 40, 2, 3, [("causal",), ("window", 1000), ("and",), ("prefix", 70), ("or",)]),
    (1, [70000], 5, 1, 64, 32, 64, 1, 4, [("causal",)]),                                   # 2188 blocks
    (1, [9000], 40, 2, 128, 64, 7, 0, 1, [("causal",)]),                                   # 20 heads a group
    (65, [700] * 65, 2, 1, 64, 64, 4, 1, 1, [("causal",)]),
    (40, list(range(100, 4100, 100)), 16, 8, 128, 64, 6, 1, 1, [("causal",)]),             # more rows than CTAs share
])
def test_choice_of_one_query(fa, B, lens, Hq, Hkv, d, page, keep, first, last, spec):
    src, q, box, table, _ = paged_case(fa, B, lens, Hq, Hkv, d, page, B + keep, spec)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    bm = fa.select_blocks(src, q[:, :, 0].contiguous(), box, keep, first, last, page_table=table, status=status)
    assert fa.check_status(status) == fa.OK
    nk = src.c.nk
    same_tables(bm, ref.select(src.tables()["block_class"], q, ref.Paged(box, table, nk), keep, first, last, 1))
    # the same from contiguous bounds
    held = box[table.clamp(min=0).long()].transpose(1, 2).contiguous()
    dense = fa.select_blocks(src, q, held, keep, first, last, out=bm)
    assert dense is bm
    same_tables(bm, ref.select(src.tables()["block_class"], q, ref.Dense(held), keep, first, last, 1))
    assert bm.c.row_max == min(keep, nk)


@pytest.mark.parametrize("B,Q,Hq,Hkv,d,bq,bk,keep,first,last,spec", [
    (1, 2, 1, 1, 64, 128, 128, 1, 0, 1, [("causal",)]),
    (2, 1000, 4, 4, 64, 128, 128, 3, 1, 1, [("causal",)]),
    (1, 1500, 6, 2, 128, 64, 128, 4, 0, 1, [("causal",)]),
    (2, 700, 8, 2, 64, 16, 32, 5, 1, 1, [("causal",), ("window", 400), ("and",)]),
    (1, 2500, 2, 1, 64, 128, 32, 9, 1, 4, [("causal",)]),
    (1, 300, 3, 3, 128, 7, 5, 11, 2, 1, [("causal",), ("prefix", 33), ("or",)]),
    (2, 640, 16, 2, 64, 128, 64, 2, 0, 0, [("true",)]),
    (3, 130, 2, 2, 64, 128, 128, 1, 0, 0, [("causal",)]),
    (1, 300, 40, 2, 64, 128, 32, 3, 0, 1, [("causal",)]),        # 20 heads a group, few rows: each head's sums for itself
    (1, 5000, 20, 2, 128, 16, 128, 6, 1, 1, [("causal",)]),      # 10 heads a group, many rows: divisions of 8 at most
    (1, 1100, 2, 1, 64, 1, 64, 3, 0, 1, [("causal",)]),          # a query a row
    (2, 1300, 4, 4, 128, 16, 32, 6, 1, 2, [("causal",)]),
    (4, 700, 6, 2, 64, 5, 33, 4, 0, 1, [("causal",), ("window", 300), ("and",)]),
])
def test_choice_of_query_blocks(fa, B, Q, Hq, Hkv, d, bq, bk, keep, first, last, spec):
    rule = fa.make_mask_rule(spec)
    src = fa.create_block_mask(rule, B, Hq, Q, Q, bq, bk)
    q, k = bf((B, Hq, Q, d), Q, spread=False), bf((B, Hkv, Q, d), Q + 1)
    box = fa.key_bounds(k, bk)
    bm = fa.select_blocks(src, q, box, keep, first, last)
    same_tables(bm, ref.select(src.tables()["block_class"], q, ref.Dense(box), keep, first, last, bq))


@pytest.mark.parametrize("sorted_ids", [True, False])
def test_choice_within_documents(fa, sorted_ids):
    N = 900
    ids = torch.arange(N, device="cuda") // 211 if sorted_ids else (torch.arange(N, device="cuda") // 100) % 3
    doc = torch.stack([ids, ids.flip(0) if not sorted_ids else ids // 2]).to(torch.int32).contiguous()
    rule = fa.make_mask_rule([("causal",), ("doc",), ("and",)], doc_ids=doc)
    src = fa.create_block_mask(rule, 2, 4, N, N, 64, 64, keep=[doc])
    q, k = bf((2, 4, N, 64), 1, spread=False), bf((2, 2, N, 64), 2)
    box = fa.key_bounds(k, 64)
    cls = ref.select(src.tables()["block_class"], q, ref.Dense(box), 2, 0, 1, 64)
    bm = fa.select_blocks(src, q, box, 2, 0, 1)
    same_tables(bm, cls)
    # the forward reads the document runs through the chosen mask too
    v = bf((2, 2, N, 64), 3, spread=False)
    o, lse = fa.flex_forward(q, k, v, bm, out_dtype=torch.float32)
    i = np.arange(N)
    pairs = (i[:, None] >= i) & (doc.cpu().numpy()[:, :, None] == doc.cpu().numpy()[:, None])
    check(o, lse, *ref.attention(q, k, v, ref.allowed(cls, pairs, 64, 64), 64**-0.5))


@pytest.mark.parametrize("Q,off,page,keep", [(1, 40000, 32, 20), (200, 36000, 32, 20), (130, 4000, 128, 3), (64, 1, 64, 1), (MANY, 9000, 32, 20)])
def test_choice_of_a_chunk_over_pages(fa, Q, off, page, keep):
    lens = [off + Q, max(off // 3, 1) + Q]
    bq = 1 if Q in (1, MANY) else 128
    src, q, box, table, _ = paged_case(fa, 2, lens, 6, 2, 64, page, Q, Q=Q, bq=bq)
    bm = fa.select_blocks(src, q, box, keep, 0, 1, page_table=table)
    same_tables(bm, ref.select(src.tables()["block_class"], q, ref.Paged(box, table, src.c.nk), keep, 0, 1, bq))


@pytest.mark.parametrize("Q", [1, 3, 300, MANY])
def test_ties_go_to_the_lower_column(fa, Q):
    N = 64 * 50
    off = torch.full((1,), N - Q, dtype=torch.int32, device="cuda")
    src = fa.create_block_mask(fa.make_mask_rule([("causal",)], q_offset=off), 1, 2, Q, N, block_of(Q), 64)
    q = bf((1, 2, Q, 128), 4, spread=False)
    some = boxes((1, 1, 3, 2, 128), 5)
    box = some[:, :, torch.arange(50, device="cuda") % 3].contiguous()            # three boxes, over and over
    for keep in (1, 7, 20, 40):
        bm = fa.select_blocks(src, q, box, keep, 0, 1)
        same_tables(bm, ref.select(src.tables()["block_class"], q, ref.Dense(box), keep, 0, 1, block_of(Q)))
    zero = torch.zeros_like(q)
    bm = fa.select_blocks(src, zero, box, 9, 2, 1)                                  # every score is 0
    same_tables(bm, ref.select(src.tables()["block_class"], zero, ref.Dense(box), 9, 2, 1, block_of(Q)))


@pytest.mark.parametrize("Q,n,Bk", [(1, 300, 16), (1, 2200, 8), (130, 300, 16), (70, 4200, 4), (200, 4200, 4), (MANY, 300, 16), (MANY, 2200, 8)])
def test_ties_of_long_rows(fa, Q, n, Bk):
    # rows that more than one warp searches, with more equal scores than are sorted at hand: in shared memory and in the workspace
    off = torch.full((1,), n * Bk - Q, dtype=torch.int32, device="cuda")
    src = fa.create_block_mask(fa.make_mask_rule([("causal",)], q_offset=off), 1, 2, Q, n * Bk, block_of(Q), Bk)
    q = bf((1, 2, Q, 64), 14, spread=False)
    some = boxes((1, 1, 5, 2, 64), 15)
    box = some[:, :, torch.arange(n, device="cuda") % 5].contiguous()
    box[:, :, 17] = some[:, :, 0] * 2
    for keep in (3, n // 7, n // 2, n - 3):
        bm = fa.select_blocks(src, q, box, keep, 1, 1)
        same_tables(bm, ref.select(src.tables()["block_class"], q, ref.Dense(box), keep, 1, 1, block_of(Q)))


# rows whose keys fill about 48 KB of shared memory, which a kernel gets without asking, together with what it has of its own
@pytest.mark.parametrize("Q,n,Bk", [(1, 2500, 8), (1, 9700, 4), (1, 9900, 4), (1, 10100, 4), (MANY, 1180, 4), (MANY, 1240, 4), (MANY, 1290, 4), (MANY, 1320, 4)])
def test_rows_that_fill_shared_memory(fa, Q, n, Bk):
    N = n * Bk
    off = torch.tensor([N - Q], dtype=torch.int32, device="cuda")
    src = fa.create_block_mask(fa.make_mask_rule([("causal",)], q_offset=off), 1, 2, Q, N, 1, Bk)
    q, box = bf((1, 2, Q, 64), n, spread=False), boxes((1, 1, n, 2, 64), n + 1)
    bm = fa.select_blocks(src, q, box, 40)
    same_tables(bm, ref.select(src.tables()["block_class"], q, ref.Dense(box), 40, 1, 1, src.c.bq))


@pytest.mark.parametrize("Q", [1, 200, MANY])
def test_scores_that_32_bits_cannot_tell_apart(fa, Q):
    # large parts that cancel, and a small one that decides: 1 / 65536 of a channel against sums of 2^14
    N, d = 64 * 40, 64
    off = torch.full((1,), N - Q, dtype=torch.int32, device="cuda")
    src = fa.create_block_mask(fa.make_mask_rule([("causal",)], q_offset=off), 1, 1, Q, N, block_of(Q), 64)
    q = torch.ones(1, 1, Q, d, device="cuda")
    q[..., 0], q[..., 1], q[..., 2] = 16384, 16384, 1.0 / 1024
    q = q.to(BF)
    box = boxes((1, 1, 1, 2, d), 8).expand(1, 1, 40, 2, d).clone()
    box[..., 0, :2], box[..., 1, 0], box[..., 1, 1] = -300, 200, -200
    box[..., 1, 2] = torch.randperm(40, generator=gen(9), device="cuda").to(BF) / 256
    box[..., 0, 2] = -1
    for keep in (2, 11, 30):
        bm = fa.select_blocks(src, q, box, keep, 0, 1)
        cls = ref.select(src.tables()["block_class"], q, ref.Dense(box), keep, 0, 1, block_of(Q))
        same_tables(bm, cls)


@pytest.mark.parametrize("Q", [1, 140, MANY])
def test_queries_far_apart_in_magnitude(fa, Q):
    # heads and rows of 2^-20 .. 2^20: a sum in 32 bits would lose the small ones, which the choice can hang on
    N, d, Hq = 64 * 30, 64, 4
    off = torch.full((2,), N - Q, dtype=torch.int32, device="cuda")
    src = fa.create_block_mask(fa.make_mask_rule([("causal",)], q_offset=off), 2, Hq, Q, N, block_of(Q), 64)
    q = bf((2, Hq, Q, d), 11, spread=False).float()
    q *= torch.exp2(torch.randint(-20, 21, (2, Hq, Q, 1), generator=gen(12), device="cuda").float())
    q = q.to(BF)
    box = boxes((2, 1, 30, 2, d), 13)
    box[:, :, 1::2] = box[:, :, 0::2]                     # pairs of equal blocks
    box[:, :, 1::2, 1, 5] += 0.0625
    for keep in (3, 8, 15, 22):
        bm = fa.select_blocks(src, q, box, keep, 0, 1)
        want = ref.select(src.tables()["block_class"], q, ref.Dense(box), keep, 0, 1, block_of(Q))
        if Q != MANY:
            same_tables(bm, want)
            continue
        # A row of four queries alone: where the large ones are negative in channel 5, two blocks of a pair differ by 0.0625 times a query of
        # 2^-20 in scores of 2^20 and more, 2^-44 of their magnitudes or less. That is under the 2^-28 that the choice promises to tell
        # apart, so there either block of a pair may be taken: the scores of the blocks that differ lie within 2^-28 of their magnitudes.
        got = bm.tables()["block_class"].cpu().numpy()
        same_tables(bm, got)
        assert np.array_equal((got > 0).sum(-1), (want > 0).sum(-1))
        qs, bs = q.double().cpu().numpy(), box.double().cpu().numpy()
        for b, r in np.argwhere((got != want).any(-1)[:, 0]):
            score = ref.scores(qs[b, :, r], bs[b, 0])
            size = ref.scores(np.abs(qs[b, :, r]), np.abs(bs[b, 0]).max(1, keepdims=True).repeat(2, 1))
            off = np.flatnonzero((got != want)[b, 0, r])
            assert np.ptp(score[off]) <= 2.0**-28 * size[off].max()


@pytest.mark.parametrize("Q", [1, 150, MANY])
def test_nan_infinite_and_huge_scores(fa, Q):
    N, d = 64 * 20, 64
    off = torch.full((1,), N - Q, dtype=torch.int32, device="cuda")
    src = fa.create_block_mask(fa.make_mask_rule([("causal",)], q_offset=off), 1, 2, Q, N, block_of(Q), 64)
    q = bf((1, 2, Q, d), 21, spread=False)
    q[..., 0] = q[..., 0].abs() + 0.1                     # no zero against an infinity
    base = boxes((1, 1, 20, 2, d), 22)
    nan, inf, huge, low = (base.clone() for _ in range(4))
    nan[0, 0, 4, :, 9] = math.nan
    nan[0, 0, 7, 1, 9] = math.nan
    inf[0, 0, 3, 1, 0] = math.inf
    inf[0, 0, 8, 1, 0] = inf[0, 0, 11, 1, 0] = math.inf
    huge[0, 0, :, 1, :4] = torch.finfo(BF).max            # sums past fp32's range, not past 64 bits'
    huge[0, 0, 5, 1, 3] = 0
    low[0, 0, :, 0, :] = torch.finfo(BF).min
    for box in (nan, inf, huge, low):
        for keep in (1, 2, 3, 6, 19):
            bm = fa.select_blocks(src, q, box, keep, 0, 1)
            same_tables(bm, ref.select(src.tables()["block_class"], q, ref.Dense(box), keep, 0, 1, block_of(Q)))


@pytest.mark.parametrize("Q", [1, 150, MANY])
def test_tiny_scores(fa, Q):
    N, d = 64 * 20, 64
    off = torch.full((1,), N - Q, dtype=torch.int32, device="cuda")
    src = fa.create_block_mask(fa.make_mask_rule([("causal",)], q_offset=off), 1, 1, Q, N, block_of(Q), 64)
    q = (bf((1, 1, Q, d), 31, spread=False).float() * 2.0**-70).to(BF)
    box = (boxes((1, 1, 20, 2, d), 32).float() * 2.0**-75).to(BF)      # products of 2^-145: under fp32's normal range
    for keep in (2, 9):
        bm = fa.select_blocks(src, q, box, keep, 0, 1)
        same_tables(bm, ref.select(src.tables()["block_class"], q, ref.Dense(box), keep, 0, 1, block_of(Q)))


@pytest.mark.parametrize("Q", [1, 100, MANY])
def test_missing_pages_rank_lowest_and_are_reported(fa, Q):
    src, q, box, table, _ = paged_case(fa, 2, [1000, 900], 4, 2, 64, 64, 41, Q=Q, bq=64 if Q == 100 else 1)
    table[0, 3], table[1, 5], table[1, 0] = -1, 10**6, -7
    for keep in (4, 14):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        bm = fa.select_blocks(src, q, box, keep, 0, 1, page_table=table, status=status)
        assert fa.check_status(status) == fa.ERR_DEVICE_CHECK
        same_tables(bm, ref.select(src.tables()["block_class"], q, ref.Paged(box, table, src.c.nk), keep, 0, 1, src.c.bq))


@pytest.mark.parametrize("Q", [1, 100, MANY])
def test_pages_are_not_looked_at_where_nothing_is_scored(fa, Q):
    src, q, box, table, _ = paged_case(fa, 2, [1000, 900], 4, 2, 64, 64, 42, Q=Q, bq=64 if Q == 100 else 1)
    bad = torch.full_like(table, 10**6)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    bm = fa.select_blocks(src, q, box, 3, 1, 2, page_table=bad, status=status)
    assert fa.check_status(status) == fa.OK
    same_tables(bm, ref.select(src.tables()["block_class"], q, ref.Paged(box, table, src.c.nk), 3, 1, 2, src.c.bq))


def test_a_mask_built_anew_for_other_sizes(fa):
    src = fa.create_block_mask(fa.make_mask_rule([("causal",)]), 1, 4, 512, 512, 64, 64)
    for n in (512, 300, 129):
        fa.recreate_block_mask(src, fa.make_mask_rule([("causal",)]), 1, 4, n, n, 64, 64)
        q, box = bf((3, 4, n, 64), n, spread=False), boxes((3, 2, (n + 63) // 64, 2, 64), n + 1)
        bm = fa.select_blocks(src, q, box, 3)
        same_tables(bm, ref.select(src.tables()["block_class"], q, ref.Dense(box), 3, 1, 1, 64))


def test_bounds_past_32_bit_offsets(fa):
    # 1.1 million pages of 8 heads and 2 x 128 channels: 2.25 G elements, the last pages lie past 2^31
    P, Hkv, d, page, n = 1_100_000, 8, 128, 64, 60
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("memory")
    box = torch.empty(P, Hkv, 2, d, dtype=BF, device="cuda")
    few = boxes((n, Hkv, 2, d), 51)
    ids = torch.arange(P - n, P, device="cuda").flip(0)
    box[ids] = few
    off = torch.tensor([n * page - 1], dtype=torch.int32, device="cuda")
    src = fa.create_block_mask(fa.make_mask_rule([("causal",)], q_offset=off), 1, 16, 1, n * page, 1, page)
    q = bf((1, 16, 1, d), 52, spread=False)
    bm = fa.select_blocks(src, q, box, 9, 1, 1, page_table=ids.to(torch.int32).view(1, n))
    same_tables(bm, ref.select(src.tables()["block_class"], q, ref.Dense(few.transpose(0, 1)[None].contiguous()), 9, 1, 1, 1))


# ---------------------------------------------------------------------------------------------- attention over the choice
def check(o, lse, o_ref, lse_ref):
    o, lse = o.double().cpu(), lse.double().cpu()
    empty = lse_ref.isneginf()
    assert torch.equal(lse.isneginf(), empty) and bool(o.isfinite().all())
    err = (o - o_ref).abs()
    assert float(err.max()) <= O_MAX and float(err.mean()) <= O_MEAN
    if not bool(empty.all()):
        assert float((lse - lse_ref)[~empty].abs().max()) <= LSE_MAX


def gather(pages, table, n):
    return pages[table.clamp(min=0).long()].transpose(1, 2).flatten(2, 3)[:, :, :n]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B,lens,Hq,Hkv,d,page,keep,first,last,cap", [
    (1, [1], 2, 1, 64, 32, 1, 0, 1, 0.0),
    (3, [2000, 64, 700], 8, 2, 128, 64, 6, 1, 2, 0.0),
    (1, [9000], 4, 4, 64, 32, 17, 0, 1, 20.0),
    (2, [5000, 4999], 16, 1, 128, 128, 12, 1, 1, 0.0),
    (2, [30000, 7], 32, 8, 128, 64, 32, 1, 2, 0.0),
    (40, [700] * 40, 16, 8, 64, 64, 3, 0, 1, 0.0),
])
def test_decode_over_the_choice(fa, fp8, B, lens, Hq, Hkv, d, page, keep, first, last, cap):
    src, q, box, table, off = paged_case(fa, B, lens, Hq, Hkv, d, page, 60 + keep)
    P = box.shape[0]
    (k, ks), (v, vs) = cache(P, Hkv, page, d, 61, fp8), cache(P, Hkv, page, d, 62, fp8)
    cls = ref.select(src.tables()["block_class"], q, ref.Paged(box, table, src.c.nk), keep, first, last, 1)
    bm = fa.select_blocks(src, q, box, keep, first, last, page_table=table)
    sc = fa.make_score_rule(softcap=cap)
    n = src.c.kv_len
    pairs = np.arange(n) <= off.cpu().numpy()[:, None, None]
    scale = 0.3 / math.sqrt(d)
    want = ref.attention(q, gather(values(k, ks), table, n), gather(values(v, vs), table, n), ref.allowed(cls, pairs, 1, page), scale, cap)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    if fp8:
        o, lse = fa.flex_decode_fp8(q[:, :, 0], k, v, ks, vs, table, bm, sc, scale, status=status, out_dtype=torch.float32)
    else:
        o, lse = fa.flex_decode(q[:, :, 0].contiguous(), k, v, table, bm, sc, scale, status=status, out_dtype=torch.float32)
        o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
        assert fa.flex_decode_noalloc(q[:, :, 0].contiguous(), k, v, table, bm, sc, scale, o2, lse2) == fa.OK
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert fa.check_status(status) == fa.OK
    # values of magnitude up to 8: the tolerance of N(0, 1) values grows with them
    top = max(1.0, float(want[0].abs().max()))
    check(o / top, lse, want[0][:, :, 0] / top, want[1][:, :, 0])


def test_decode_over_an_empty_choice(fa):
    # a request whose position sees nothing (a window of a later prefix): no block to choose, O = 0 and LSE = -inf
    src, q, box, table, off = paged_case(fa, 2, [300, 200], 4, 2, 64, 32, 71)
    off[1] = -1
    src = fa.create_block_mask(fa.make_mask_rule([("causal",)], q_offset=off), 2, 4, 1, src.c.kv_len, 1, 32)
    k, v = (cache(box.shape[0], 2, 32, 64, s, False)[0] for s in (72, 73))
    bm = fa.select_blocks(src, q, box, 4, 1, 1, page_table=table)
    o, lse = fa.flex_decode(q[:, :, 0].contiguous(), k, v, table, bm)
    assert not o[1].any() and bool(lse[1].isneginf().all()) and bool(lse[0].isfinite().all())


GRAD = 2e-2  # of a gradient's largest magnitude, as for the backward over any mask


@pytest.mark.parametrize("B,N,Hq,Hkv,d,block,keep,first,last,cap,window", [
    (1, 700, 4, 2, 64, 128, 3, 1, 1, 0.0, 0),
    (2, 513, 3, 3, 128, 128, 2, 0, 1, 0.0, 0),
    (1, 600, 8, 2, 128, 64, 3, 0, 1, 20.0, 0),
    (1, 900, 6, 2, 64, 128, 2, 0, 0, 0.0, 300),      # rows may lose the block of their own position
    (1, 1, 2, 1, 64, 128, 1, 0, 1, 0.0, 0),
    (1, 1025, 16, 2, 128, 128, 4, 1, 2, 0.0, 0),
    (2, 1500, 8, 4, 64, 128, 10, 1, 1, 0.0, 0),      # columns of a key block shared by two CTAs
    (2, 1400, 8, 8, 64, 128, 10, 1, 1, 0.0, 0),      # and by none
])
def test_forward_and_backward_over_the_choice(fa, B, N, Hq, Hkv, d, block, keep, first, last, cap, window):
    spec = [("causal",)] + ([("window", window), ("and",)] if window else [])
    src = fa.create_block_mask(fa.make_mask_rule(spec), B, Hq, N, N, block, block)
    q, k, v, do = (bf((B, h, N, d), 80 + i, spread=False) for i, h in enumerate((Hq, Hkv, Hkv, Hq)))
    box = fa.key_bounds(k, block)
    cls = ref.select(src.tables()["block_class"], q, ref.Dense(box), keep, first, last, block)
    bm = fa.select_blocks(src, q, box, keep, first, last)
    same_tables(bm, cls)
    i = np.arange(N)
    pairs = (i[:, None] >= i) & ((i[:, None] - i < window) if window else True)
    want = ref.attention(q, k, v, ref.allowed(cls, pairs[None], block, block), d**-0.5, cap, do)
    sc = fa.make_score_rule(softcap=cap)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse = fa.flex_forward(q, k, v, bm, sc, status=status, out_dtype=torch.float32)
    check(o, lse, *want[:2])
    o2, lse2 = fa.flex_forward(q, k, v, bm, sc, force_mma=True, out_dtype=torch.float32)
    check(o2, lse2, *want[:2])
    if block == 128:
        o3, lse3 = fa.flex_forward_split(q, k, v, bm, sc, chunk_blocks=2, out_dtype=torch.float32)
        check(o3, lse3, *want[:2])
    # With one key P = 1 and dS = <dO, V> - <dO, O> is 0: two fp32 sums of the same d products in other orders, each off by at most
    # d 2^-24 of their magnitudes; dQ and dK (a sum over the group's heads) multiply that by scale times K or Q.
    rest = 0.0
    if N == 1:
        most = float((do.double().abs() * v.double().abs().repeat_interleave(Hq // Hkv, 1)).sum(-1).max())
        rest = 2 * d * 2.0**-24 * most * d**-0.5 * max(float(q.abs().max()), float(k.abs().max())) * (Hq // Hkv)
    for got, w in zip(fa.flex_backward(q, k, v, o, lse, do, bm, sc, status=status), want[2:]):
        assert float((got.double().cpu() - w).abs().max()) <= max(GRAD * max(float(w.abs().max()), 1e-6), rest)
    assert fa.check_status(status) == fa.OK
    host = [x.cpu().pin_memory() for x in (q, k, v)]
    oh, lh = torch.empty(o.shape).pin_memory(), torch.empty(lse.shape).pin_memory()
    fa.flex_forward_host(*host, bm, sc, out=oh, lse=lh)
    torch.cuda.synchronize()
    assert torch.equal(oh, o.cpu()) and torch.equal(lh, lse.cpu())


def blockwise(q, k, v, do, cls, scale):
    """Gradients in 64 bits of one causal sequence over 128 x 128 blocks, a query block of a head at a time."""
    g, N = q.shape[0] // k.shape[0], q.shape[1]
    q, k, v, do = (x.double() for x in (q, k, v, do))
    dq, dk, dv = (torch.zeros_like(x) for x in (q, k, v))
    for h in range(q.shape[0]):
        for r in range(cls.shape[1]):
            i = torch.arange(r * 128, min(N, r * 128 + 128), device="cuda")
            j = torch.cat([torch.arange(c * 128, min(N, c * 128 + 128), device="cuda") for c in np.flatnonzero(cls[h // g, r])])
            kj, vj = k[h // g, j], v[h // g, j]
            p = (q[h, i] @ kj.T * scale).masked_fill(j[None] > i[:, None], -math.inf).softmax(-1)
            ds = do[h, i] @ vj.T
            ds = p * (ds - (p * ds).sum(-1, keepdim=True)) * scale
            dq[h, i] = ds @ kj
            dk[h // g, j] += ds.T @ q[h, i]
            dv[h // g, j] += p.T @ do[h, i]
    return dq, dk, dv


# columns of a key block that four CTAs share, two, none; more key blocks than a CTA puts in order of length
@pytest.mark.parametrize("N,Hq,Hkv,d,keep", [(6000, 8, 2, 64, 9), (6100, 16, 4, 128, 14), (3000, 8, 8, 64, 8), (41000, 2, 1, 64, 4)])
def test_gradients_of_long_columns(fa, N, Hq, Hkv, d, keep):
    src = fa.create_block_mask(fa.make_mask_rule([("causal",)]), 1, Hq, N, N, 128, 128)
    q, k, v, do = (bf((1, h, N, d), 180 + i, spread=False) for i, h in enumerate((Hq, Hkv, Hkv, Hq)))
    bm = fa.select_blocks(src, q, fa.key_bounds(k), keep)
    o, lse = fa.flex_forward(q, k, v, bm)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = fa.flex_backward(q, k, v, o, lse, do, bm, status=status)
    again = fa.flex_backward(q, k, v, o, lse, do, bm)
    assert fa.check_status(status) == fa.OK and all(torch.equal(x, y) for x, y in zip(got, again))
    for x, w in zip(got, blockwise(q[0], k[0], v[0], do[0], bm.tables()["block_class"][0].cpu().numpy(), d**-0.5)):
        assert float((x[0].double() - w).abs().max()) <= GRAD * float(w.abs().max())


@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (16, 16)])
def test_what_follows_a_backward_reads_whole_gradients(fa, Hq, Hkv):
    # captured with the copies that follow it, and eagerly on a side stream: dQ's kernel starts before that of dK and dV has ended
    N, d = 2500, 128
    src = fa.create_block_mask(fa.make_mask_rule([("causal",)]), 1, Hq, N, N, 128, 128)
    q, k, v, do = (bf((1, h, N, d), 280 + i, spread=False) for i, h in enumerate((Hq, Hkv, Hkv, Hq)))
    bm = fa.select_blocks(src, q, fa.key_bounds(k), 5)
    o, lse = fa.flex_forward(q, k, v, bm)
    want = fa.flex_backward(q, k, v, o, lse, do, bm)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(3):
            got = [x.clone() for x in fa.flex_backward(q, k, v, o, lse, do, bm)]
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        grads = fa.flex_backward(q, k, v, o, lse, do, bm)
        copies = [x.clone() for x in grads]
        for x in grads:
            x.fill_(math.nan)               # the next replay has to write all of them again
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(copies, want))


def test_gradient_over_the_choice_against_differences(fa):
    # the choice held fixed, as training does: f = sum(dout * O) along a direction
    N, d = 300, 64
    src = fa.create_block_mask(fa.make_mask_rule([("causal",)]), 1, 2, N, N, 64, 64)
    q, k, v, do = (bf((1, h, N, d), 90 + i, spread=False) for i, h in enumerate((2, 1, 1, 2)))
    bm = fa.select_blocks(src, q, fa.key_bounds(k, 64), 2, 0, 1)
    cls = bm.tables()["block_class"].cpu().numpy()
    o, lse = fa.flex_forward(q, k, v, bm, out_dtype=torch.float32)
    grads = fa.flex_backward(q, k, v, o, lse, do, bm)
    i = np.arange(N)
    ok = ref.allowed(cls, (i[:, None] >= i)[None], 64, 64)
    f = lambda *x: float((ref.attention(*x, ok, d**-0.5)[0] * do.double().cpu()).sum())  # noqa: E731
    at = [x.double().cpu() for x in (q, k, v)]
    for w in range(3):
        u = bf(at[w].shape, 95 + w, spread=False).double().cpu()
        h = 1e-4
        up, down = ([x + s * h * u if j == w else x for j, x in enumerate(at)] for s in (1, -1))
        slope, got = (f(*up) - f(*down)) / (2 * h), float((grads[w].double().cpu() * u).sum())
        # each element is off by GRAD of the largest at most, in no one direction
        assert abs(got - slope) <= GRAD * float(grads[w].abs().max()) * math.sqrt(u.numel())


@pytest.mark.parametrize("page,Hq,Hkv,Q", [(128, 8, 2, 200), (128, 4, 4, 20), (64, 8, 2, 130)])
def test_chunk_over_the_choice(fa, page, Hq, Hkv, Q):
    d, lens = 64, [1500, 900]
    src, q, box, table, off = paged_case(fa, 2, lens, Hq, Hkv, d, page, 100 + Q, Q=Q, bq=128)
    P, n = box.shape[0], src.c.kv_len
    cls = ref.select(src.tables()["block_class"], q, ref.Paged(box, table, src.c.nk), 4, 1, 2, 128)
    bm = fa.select_blocks(src, q, box, 4, 1, 2, page_table=table)
    same_tables(bm, cls)
    pairs = np.arange(n) <= (off.cpu().numpy()[:, None] + np.arange(Q))[..., None]
    for fp8 in (False, True):
        (k, ks), (v, vs) = cache(P, Hkv, page, d, 101, fp8), cache(P, Hkv, page, d, 102, fp8)
        want = ref.attention(q, gather(values(k, ks), table, n), gather(values(v, vs), table, n), ref.allowed(cls, pairs, 128, page), 0.3 / math.sqrt(d))
        top = max(1.0, float(want[0].abs().max()))
        runs = [fa.flex_forward_paged_fp8(q, k, v, ks, vs, table, bm, n, scale=0.3 / math.sqrt(d), chunk_blocks=c, out_dtype=torch.float32)
                for c in ((0, -1, 3) if page == 128 else (0,))] if fp8 else [fa.flex_forward_paged(q, k, v, table, bm, n, scale=0.3 / math.sqrt(d), out_dtype=torch.float32)]
        for o, lse in runs:
            check(o / top, lse, want[0] / top, want[1])


# ---------------------------------------------------------------------------------------------- as a program runs them
def serve(fa, B, Hq, Hkv, d, page, fp8, steps_max, seed):
    """A cache and the calls of one decode step: append, bounds, mask, choice, attention."""
    width = (steps_max + page - 1) // page
    P = B * width + 1
    pools = []
    for _ in range(2):
        pools.append(torch.zeros(P, Hkv, page, d, dtype=torch.uint8, device="cuda").view(ref.F8) if fp8 else torch.zeros(P, Hkv, page, d, dtype=BF, device="cuda"))
    scales = [torch.zeros(P, Hkv, page // 32, device="cuda") for _ in range(2)]
    table = torch.randperm(P, generator=gen(seed), device="cuda")[:B * width].to(torch.int32).view(B, width)
    bounds = torch.zeros(P, Hkv, 2, d, dtype=BF, device="cuda")
    freq = 10000.0 ** (-2 * torch.arange(d // 2, device="cuda") / d)
    return dict(k=pools[0], v=pools[1], ks=scales[0], vs=scales[1], table=table, bounds=bounds, rule=fa.make_qk_rule(inv_freq=freq), width=width, page=page, fp8=fp8,
                Hq=Hq, Hkv=Hkv, d=d, B=B)


def append(fa, s, rows, off, n_new):
    x = rows.split([s["Hq"], s["Hkv"], s["Hkv"]], dim=2)
    N = rows.shape[1]
    if s["fp8"]:
        q = fa.kv_append_fp8(*x, s["k"], s["v"], s["ks"], s["vs"], s["table"], s["rule"], q_offset=off, n_new=n_new)
        fa.kv_bounds_fp8(s["k"], s["ks"], s["bounds"], s["table"], N, q_offset=off, n_new=n_new)
    else:
        q = fa.kv_append(*x, s["k"], s["v"], s["table"], s["rule"], q_offset=off, n_new=n_new)
        fa.kv_bounds(s["k"], s["bounds"], s["table"], N, q_offset=off, n_new=n_new)
    return q


def attend(fa, s, q, off, keep, workspace=None, masks=None):
    src = fa.create_block_mask(fa.make_mask_rule([("causal",)], q_offset=off), s["B"], s["Hq"], 1, s["width"] * s["page"], 1, s["page"], keep=[off],
                               buf=masks[0].buf if masks else None)
    bm = fa.select_blocks(src, q, s["bounds"], keep, 1, 2, page_table=s["table"], out=masks[1] if masks else None, workspace=workspace)
    if s["fp8"]:
        return bm, *fa.flex_decode_fp8(q[:, :, 0], s["k"], s["v"], s["ks"], s["vs"], s["table"], bm, out_dtype=torch.float32)
    return bm, *fa.flex_decode(q[:, :, 0].contiguous(), s["k"], s["v"], s["table"], bm, out_dtype=torch.float32)


@pytest.mark.parametrize("fp8", [False, True])
def test_a_request_served(fa, fp8):
    # a prompt, then tokens one at a time across page borders; each step against the cache's own values
    B, Hq, Hkv, d, page, keep = 3, 8, 2, 64, 32, 5
    s = serve(fa, B, Hq, Hkv, d, page, fp8, 500, 7)
    lens = torch.tensor([300, 1, 95], dtype=torch.int32, device="cuda")
    append(fa, s, bf((B, 300, Hq + 2 * Hkv, d), 1, spread=False), torch.zeros_like(lens), lens)
    for step in range(4):
        q = append(fa, s, bf((B, 1, Hq + 2 * Hkv, d), 2 + step, spread=False), lens, None)
        x = values(s["k"], s["ks"] if fp8 else None)
        held = s["bounds"].double()
        for b in range(B):
            for t in range(int(lens[b]) // page + 1):
                pid, n = int(s["table"][b, t]), min(page, int(lens[b]) + 1 - t * page)
                assert torch.equal(held[pid, :, 0], x[pid, :, :n].amin(1)) and torch.equal(held[pid, :, 1], x[pid, :, :n].amax(1))
        bm, o, lse = attend(fa, s, q, lens, keep)
        n = s["width"] * page
        pairs = np.arange(n) <= lens.cpu().numpy()[:, None, None]
        src = np.zeros((B, 1, 1, s["width"]), np.uint8)
        for b in range(B):
            last = int(lens[b])
            src[b, 0, 0, :last // page + 1] = 2
            if last % page != page - 1:
                src[b, 0, 0, last // page] = 1
        cls = ref.select(torch.from_numpy(src), q, ref.Paged(s["bounds"], s["table"], s["width"]), keep, 1, 2, 1)
        same_tables(bm, cls)
        k, v = (gather(values(s[p], s[p + "s"] if fp8 else None), s["table"], n) for p in "kv")
        want = ref.attention(q, k, v, ref.allowed(cls, pairs, 1, page), d**-0.5)
        check(o, lse, want[0][:, :, 0], want[1][:, :, 0])
        lens = lens + 1


def test_two_captured_steps_on_two_streams(fa):
    B, Hq, Hkv, d, page, keep = 4, 8, 2, 64, 32, 4
    graphs, wants = [], []
    for seed in (0, 1):
        s = serve(fa, B, Hq, Hkv, d, page, seed == 1, 400, seed)
        lens = torch.tensor([350, 200, 31, 1], dtype=torch.int32, device="cuda") + seed
        append(fa, s, bf((B, 352, Hq + 2 * Hkv, d), 10 + seed, spread=False), torch.zeros_like(lens), lens)
        rows = bf((B, 1, Hq + 2 * Hkv, d), 12 + seed, spread=False)
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            want = attend(fa, s, append(fa, s, rows, lens, None), lens, keep)[1:]
            st.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=st):
                got = attend(fa, s, append(fa, s, rows, lens, None), lens, keep)
        graphs.append((graph, st, got, s, rows, lens))
        wants.append([x.clone() for x in want])
    for _ in range(20):
        for graph, st, *_ in graphs:
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    for (_, _, got, *_), want in zip(graphs, wants):
        for x, y in zip(got[1:], want):
            assert torch.equal(x, y)


def test_the_same_result_each_time(fa):
    src = fa.create_block_mask(fa.make_mask_rule([("causal",)]), 2, 8, 4000, 4000, 128, 128)
    q, k = bf((2, 8, 4000, 128), 1, spread=False), bf((2, 2, 4000, 128), 2)
    ws = torch.empty(fa.select_blocks_workspace_bytes(src, 2, 8, 2, 128), dtype=torch.uint8, device="cuda")
    bm = fa.select_blocks(src, q, fa.key_bounds(k), 6, workspace=ws)
    first = {n: t.clone() for n, t in bm.tables().items()}
    for i in range(10):
        ws.fill_(255 if i % 2 else 0)                       # nothing is read that the call did not write
        bm.buf.fill_(85)
        again = fa.select_blocks(src, q, fa.key_bounds(k), 6, workspace=ws, out=bm)
        assert again is bm
        assert all(torch.equal(t, first[n]) for n, t in bm.tables().items())


def test_a_choice_from_a_choice_is_refused_and_rows_of_one_may_be_selected(fa):
    N = 1000
    src = fa.create_block_mask(fa.make_mask_rule([("causal",)]), 1, 4, N, N, 64, 64)
    q, k = bf((1, 4, N, 64), 1, spread=False), bf((1, 2, N, 64), 2)
    box = fa.key_bounds(k, 64)
    bm = fa.select_blocks(src, q, box, 3)
    with pytest.raises(fa.FaError):
        fa.select_blocks(bm, q, box, 2)
    pos = torch.tensor([999], dtype=torch.int32, device="cuda")
    one = fa.select_rows(bm, pos)
    got, full = one.tables()["block_class"][0, :, 0], bm.tables()["block_class"][0, :, 15]
    assert torch.equal(got > 0, full > 0) and one.c.row_max == 3
    stats = fa.block_mask_stats(bm).tolist()
    assert stats[0] + stats[1] == sum(min(3, r + 1) for r in range(16)) * 2 and stats[3] == 3 and stats[5] == 32
