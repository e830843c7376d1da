"""Sums over queries that the choice of blocks hangs on: magnitudes that jump from one stretch of queries to the next, and wide groups of
heads, against the plain 64-bit form."""
import pytest
import torch

import select_ref as ref
from test_gpu_select import BF, MANY, block_of, fa, gen, same_tables  # noqa: F401 (fa is a fixture)

pytestmark = pytest.mark.gpu


def source(fa, B, Hq, Q, nk):
    """A mask in which every query sees all but the last few of nk blocks of 64 keys."""
    off = torch.full((B,), nk * 64 - Q, dtype=torch.int32, device="cuda")
    return fa.create_block_mask(fa.make_mask_rule([("causal",)], q_offset=off), B, Hq, Q, nk * 64, block_of(Q), 64, keep=[off])


@pytest.mark.parametrize("g", [46400, 65535])
def test_the_widest_groups(fa, g):  # noqa: F811
    # heads times divisions of them pass 32 bits: every head counts, the last ones most
    Q, nk, d = 2, 12, 64
    src = source(fa, 1, g, Q, nk)
    q = torch.zeros(1, g, Q, d, device="cuda")
    q[0, :, :, 0] = torch.arange(g, device="cuda")[:, None] % 3 - 1.0
    q[0, -5:, :, 1] = 1024
    q[0, g // 2, 0, 2] = -4096
    q = q.to(BF)
    box = torch.randint(1, 128, (1, 1, nk, 2, d), generator=gen(g), device="cuda").float()
    box[..., 0, :] *= -1
    box = box.to(BF)
    for keep in (2, 5):
        bm = fa.select_blocks(src, q, box, keep, 0, 1)
        same_tables(bm, ref.select(src.tables()["block_class"], q, ref.Dense(box), keep, 0, 1, block_of(Q)))


# Channel 0 holds -2^-D or +2^-D in the queries that come first and nothing afterwards, its neighbour the same and then 1. The bounds of channel 0 are
# 2^D times as large, so that both channels have a say in a score. With whole numbers of 1 ... 255 in the bounds two scores differ by 2^-16
# of their magnitudes, or are equal.
@pytest.mark.parametrize("sign", [-1.0, 1.0])
@pytest.mark.parametrize("D", [20, 30, 31, 32, 33, 40, 60])
@pytest.mark.parametrize("where,Q,d", [("rows", 128, 64), ("rows", 200, 128), ("head", MANY, 64), ("head", MANY, 128)])
def test_small_queries_before_large_ones(fa, where, Q, d, D, sign):  # noqa: F811
    nk, Hq = 30, 4
    src = source(fa, 1, Hq, Q, nk)
    q = torch.zeros(1, Hq, Q, d, device="cuda")
    small = torch.zeros(Hq, Q, dtype=torch.bool, device="cuda")
    if where == "rows":
        small[:, torch.arange(Q, device="cuda") % 64 < 32] = True     # the first half of what each half of a CTA reads
    else:
        small[0] = True
    q[0, :, :, 0] = torch.where(small, sign * 2.0**-D, 0.0)
    q[0, :, :, 1] = torch.where(small, sign * 2.0**-D, 1.0)
    q = q.to(BF)
    box = torch.zeros(1, 1, nk, 2, d, device="cuda")
    box[0, 0, :, :, :2] = torch.randint(1, 256, (nk, 1, 2), generator=gen(D), device="cuda").float() * torch.tensor([-1.0, 1.0], device="cuda")[:, None]
    box[..., 0] *= 2.0**D
    box = box.to(BF)
    for keep in (2, 7, 20):
        bm = fa.select_blocks(src, q, box, keep, 0, 1)
        same_tables(bm, ref.select(src.tables()["block_class"], q, ref.Dense(box), keep, 0, 1, block_of(Q)))


@pytest.mark.parametrize("g", [2, 6, 128, 600])
@pytest.mark.parametrize("Q", [1, 2, MANY])
def test_wide_groups_lose_nothing(fa, Q, g):  # noqa: F811
    # channel 0: 1 from one head and a little under 2^-24 from each other one, which a running 32-bit sum never takes up. A block with a bound of 1 there is ahead of a
    # rival with 1 in channel 1 and 2^-24 times two thirds of the heads in channel 2
    nk, d = 9, 64
    src = source(fa, 1, g, Q, nk)
    q = torch.zeros(1, g, Q, d, device="cuda")
    q[0, 1:, 0, 0] = 0.99 * 2.0**-24
    q[0, 0, 0, 0] = q[0, 0, 0, 1] = 1
    q[0, 0, 0, 2] = 2.0**-10
    q = q.to(BF)
    for ahead, rival in ((3, 5), (5, 3)):
        box = torch.zeros(1, 1, nk, 2, d, device="cuda")
        box[0, 0, ahead, 1, 0] = box[0, 0, rival, 1, 1] = 1
        box[0, 0, rival, 1, 2] = g * 2 / 3 * 2.0**-14
        box = box.to(BF)
        bm = fa.select_blocks(src, q, box, 2, 0, 1)
        same_tables(bm, ref.select(src.tables()["block_class"], q, ref.Dense(box), 2, 0, 1, block_of(Q)))


# Channel 0 far below its neighbour: 2^-40 in the first of the queries that a lane reads and a little under 2^-64 in all others, which a running
# 32-bit sum of them never takes up. A block whose bound there is 2^40 is ahead of a rival that takes channel 2, half as much above the large ones.
@pytest.mark.parametrize("sign", [-1.0, 1.0])
@pytest.mark.parametrize("Q,g", [(128, 1), (256, 2), (MANY, 8)])
@pytest.mark.parametrize("d", [64, 128])
def test_small_channel_beside_a_large_one(fa, Q, g, d, sign):  # noqa: F811
    nk = 9
    src = source(fa, 1, g, Q, nk)
    r = torch.arange(Q, device="cuda") % 64
    first = (torch.arange(g, device="cuda")[:, None] == 0) & ((r < 256 // d) | (Q == MANY))     # the rows of a lane's first load
    q = torch.zeros(1, g, Q, d, device="cuda")
    q[0, :, :, 0] = torch.where(first, 2.0**-40, 0.99 * 2.0**-64)
    q[0, :, :, 1] = 1
    q[0, :, :, 2] = torch.where(first, 1.0, 0.0)
    q[0, :, :, 3] = torch.where(first, 0.0, 2.0**-10)
    q = (q * torch.where(torch.arange(d, device="cuda") == 1, 1.0, sign)).to(BF)
    for ahead, rival in ((3, 5), (5, 3)):
        box = torch.zeros(1, 1, nk, 2, d, device="cuda")
        at = 0 if sign < 0 else 1
        box[0, 0, ahead, at, 0] = sign * 2.0**40
        box[0, 0, rival, at, 2] = sign
        box[0, 0, rival, at, 3] = sign * 2.0**-15                       # 2^-25 a query
        box = box.to(BF)
        bm = fa.select_blocks(src, q, box, 2, 0, 1)
        same_tables(bm, ref.select(src.tables()["block_class"], q, ref.Dense(box), 2, 0, 1, block_of(Q)))
