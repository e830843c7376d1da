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
