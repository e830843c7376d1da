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
