"""Gradients over blocks chosen under a window, whose key blocks few rows see: against 64 bits, and with the same bits each time."""
import math

import numpy as np
import pytest
import torch

from test_gpu_select import GRAD, bf, fa  # noqa: F401 (fa is a fixture)

pytestmark = pytest.mark.gpu


def gradients(q, k, v, do, cls, scale, sees):
    """In 64 bits, a query block of a head at a time; sees(i, j) the rule."""
    g, N = q.shape[0] // k.shape[0], q.shape[1]
    q, k, v, do = (x.double() for x in (q, k, v, do))
    dq, dk, dv = (torch.zeros_like(x) for x in (q, k, v))
    for h in range(q.shape[0]):
        for r in range(cls.shape[1]):
            i = torch.arange(r * 128, min(N, r * 128 + 128), device="cuda")
            j = torch.cat([torch.arange(c * 128, min(N, c * 128 + 128), device="cuda") for c in np.flatnonzero(cls[h // g, r])])
            kj, vj = k[h // g, j], v[h // g, j]
            p = (q[h, i] @ kj.T * scale).masked_fill(~sees(i[:, None], j[None]), -math.inf).softmax(-1)
            ds = do[h, i] @ vj.T
            ds = p * (ds - (p * ds).sum(-1, keepdim=True)) * scale
            dq[h, i] = ds @ kj
            dk[h // g, j] += ds.T @ q[h, i]
            dv[h // g, j] += p.T @ do[h, i]
    return dq, dk, dv


# a window with and without a prefix that all rows see, and one so wide that a cluster shares its columns; the last block of a row is always kept
@pytest.mark.parametrize("N,Hq,Hkv,d,window,prefix,keep", [(6000, 8, 2, 64, 600, 0, 4), (6000, 8, 2, 128, 600, 100, 4), (5000, 16, 2, 64, 2500, 0, 6), (3000, 4, 4, 64, 1, 0, 3)])
def test_gradients_over_a_choice_within_a_window(fa, N, Hq, Hkv, d, window, prefix, keep):  # noqa: F811
    spec = [("causal",), ("window", window), ("and",)] + ([("prefix", prefix), ("or",)] if prefix else [])
    src = fa.create_block_mask(fa.make_mask_rule(spec), 1, Hq, N, N, 128, 128)
    q, k, v, do = (bf((1, h, N, d), 480 + i, spread=False) for i, h in enumerate((Hq, Hkv, Hkv, Hq)))
    bm = fa.select_blocks(src, q, fa.key_bounds(k), keep, 0, 1 if not prefix else 2)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse = fa.flex_forward(q, k, v, bm, status=status)
    got = fa.flex_backward(q, k, v, o, lse, do, bm, status=status)
    again = fa.flex_backward(q, k, v, o, lse, do, bm)
    assert fa.check_status(status) == fa.OK and all(torch.equal(x, y) for x, y in zip(got, again))
    cls = bm.tables()["block_class"][0].cpu().numpy()
    want = gradients(q[0], k[0], v[0], do[0], cls, d**-0.5, lambda i, j: ((j <= i) & (i - j < window)) | (j < prefix))
    # Of a row with one key P = 1 and dS = <dO, V> - <dO, O> is 0 in truth: two fp32 sums of d products in other orders, and O rounded to bf16 (2^-8 of it, as V is a
    # bf16 value O is V itself there): d 2^-23 of their magnitudes, times scale and K or Q, over the group's heads
    most = float((do.double().abs() * v.double().abs().repeat_interleave(Hq // Hkv, 1)).sum(-1).max())
    rest = 2 * d * 2.0**-24 * most * d**-0.5 * max(float(q.abs().max()), float(k.abs().max())) * (Hq // Hkv)
    for x, w in zip(got, want):
        assert float((x[0].double() - w).abs().max()) <= max(GRAD * float(w.abs().max()), rest if window == 1 else 0.0)
