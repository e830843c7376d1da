"""Which of a mask's row sets each query head reads, over groups of odd and large sizes."""
import numpy as np
import pytest
import torch

import select_ref as ref
from test_gpu_select import GRAD, bf, check, fa, same_tables  # noqa: F401 (fa is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Hkv,block", [(111, 37, 128), (77, 11, 128), (195, 3, 128), (35, 7, 64), (9, 9, 128)])
def test_a_row_set_for_each_group(fa, Hq, Hkv, block):  # noqa: F811
    N, d = 300, 64
    src = fa.create_block_mask(fa.make_mask_rule([("causal",)]), 1, Hq, N, N, block, block)
    q, k, v, do = (bf((1, h, N, d), 380 + i, spread=False) for i, h in enumerate((Hq, Hkv, Hkv, Hq)))
    box = fa.key_bounds(k, block)
    cls = ref.select(src.tables()["block_class"], q, ref.Dense(box), 2, 0, 1, block)
    bm = fa.select_blocks(src, q, box, 2, 0, 1)
    same_tables(bm, cls)
    i = np.arange(N)
    want = ref.attention(q, k, v, ref.allowed(cls, (i[:, None] >= i)[None], block, block), d**-0.5, 0.0, do)
    o, lse = fa.flex_forward(q, k, v, bm, out_dtype=torch.float32)
    check(o, lse, *want[:2])
    o2, lse2 = fa.flex_forward(q, k, v, bm, force_mma=True, out_dtype=torch.float32)
    check(o2, lse2, *want[:2])
    if block == 128:
        check(*fa.flex_forward_split(q, k, v, bm, chunk_blocks=1, out_dtype=torch.float32), *want[:2])
    for got, w in zip(fa.flex_backward(q, k, v, o, lse, do, bm), want[2:]):
        assert float((got.double().cpu() - w).abs().max()) <= GRAD * float(w.abs().max())
