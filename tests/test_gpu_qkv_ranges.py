"""The attention's inputs on the GPU at sizes where a thread block takes several heads and a warp several tokens: the append of long
prompts into e4m3 pages, interleaved rotation in every append, and the weights' gradient over a full grid."""
import pytest
import torch

from block_sparse_masked_create_gb300 import fa
from tests import qkv_ref as ref
from tests.test_gpu_qkv import BF, F32, expected_block, fp8_pools, gen, make, split, tables

pytestmark = pytest.mark.gpu


def placed(rows, c, table, n_new, page, total):
    """[B, N, H, d] rows in the layout of a pool, and which slots they take."""
    B, N, H, d = rows.shape
    out = torch.zeros(total, H, page, d, dtype=rows.dtype)
    new = torch.zeros(total, H, page, dtype=torch.bool)
    for b in range(B):
        at = int(c["off"][b]) + torch.arange(int(n_new[b]))
        pid, slot = table[b, at // page].long(), at % page
        out[pid, :, slot] = rows[b, :len(at)]
        new[pid, :, slot] = True
    return out, new


@pytest.mark.parametrize("B,N,Hq,Hkv,d,rot,norm,inter,page", [
    (8, 600, 8, 8, 128, 128, True, False, 128),    # 4 heads a thread block, 2 of them loaded ahead
    (8, 600, 16, 8, 128, 48, True, True, 32),
    (8, 500, 16, 16, 64, 64, True, False, 64),     # 6 heads a thread block, 4 of them loaded ahead
    (8, 500, 17 * 2, 17, 64, 32, False, True, 64),  # heads that do not divide evenly
    (3, 1, 4, 2, 64, 32, True, True, 64), (3, 1, 32, 8, 128, 128, True, True, 128)])
def test_append_fp8_several_heads_a_block_and_interleaved(B, N, Hq, Hkv, d, rot, norm, inter, page):
    c = make(50, B, N, Hq, Hkv, d, rot, norm, inter, offset=17)
    table, total = tables(51, B, -(-(17 + 50 + N) // page))
    n_new = torch.tensor([N if b % 3 else N - N // 4 for b in range(B)], dtype=torch.int32)
    pools, scales = fp8_pools(52, total, Hkv, page, d)
    kp, vp, ks, vs = (t.clone().cuda() for t in (*pools, *scales))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    qo = fa.kv_append_fp8(*split(c), kp, vp, ks, vs, table.cuda(), c["rule"], c["cu"]["off"], n_new.cuda(), status=status)
    assert fa.check_status(status) == fa.OK
    same = fa.qk_norm_rope(*split(c), c["rule"], q_offset=c["cu"]["off"])  # the same rows, pinned by its own tests
    rows = expected_block(c, pools, scales, table, n_new, page)
    for b in range(B):
        assert torch.equal(qo[b, :, :int(n_new[b])], same[0][b, :, :int(n_new[b])])
    for z, (got, gs) in enumerate(((kp, ks), (vp, vs))):
        assert torch.equal(gs.cpu(), scales[z])
        y, new = placed(rows[1 + z][0], c, table, n_new, page, total)
        slack, _ = placed(rows[1 + z][1], c, table, n_new, page, total)
        got, s = got.cpu().float(), scales[z].double().repeat_interleave(32, -1)[..., None]
        # a new value is within half a step of e4m3 of the row's 64-bit value; all others are equal to the byte
        assert ((got.double() * s - y).abs() <= 2.0 ** -4 * y.abs() + 2.0 ** -10 * s + 2 * slack)[new].all()
        assert torch.equal(got[~new], pools[z].float()[~new])


@pytest.mark.parametrize("B,N,rot,page", [(3, 1, 32, 16), (2, 130, 64, 64)])
def test_append_bf16_interleaved(B, N, rot, page):
    Hq, Hkv, d = 4, 2, 64
    c = make(53, B, N, Hq, Hkv, d, rot, True, True, offset=3)
    table, total = tables(54, B, -(-(53 + N) // page))
    n_new = torch.full((B,), N, dtype=torch.int32)
    kp, vp = (torch.zeros(total, Hkv, page, d, dtype=BF, device="cuda") for _ in range(2))
    qo = fa.kv_append(*split(c), kp, vp, table.cuda(), c["rule"], c["cu"]["off"], n_new.cuda())
    same = fa.qk_norm_rope(*split(c), c["rule"], q_offset=c["cu"]["off"])
    assert torch.equal(qo, same[0])
    for got, want in ((kp, same[1]), (vp, same[2])):
        want, new = placed(want.cpu().transpose(1, 2), c, table, n_new, page, total)
        assert torch.equal(got.cpu()[new], want[new]) and not got.cpu()[~new].any()


@pytest.mark.parametrize("d,inter", [(128, False), (64, True)])
def test_weight_gradient_over_a_full_grid(d, inter):
    # more tokens than warps: each warp sums several items, every CTA of the grid has a row of partial sums. A row's term has the
    # roundings of its factors (64), the sum at most one for each row
    B, N, Hq, Hkv = 2, 3001, 4, 2
    c = make(55, B, N, Hq, Hkv, d, d // 2, True, inter)
    dy = [torch.randn(B, h, N, d, generator=gen(56)) for h in (Hq, Hkv, Hkv)]
    q, k, _ = split(c)
    cu = [t.cuda() for t in dy]
    both = fa.qk_norm_rope_backward(q, k, *cu, c["rule"], q_offset=c["cu"]["off"], grad_dtype=F32)
    only_k = fa.qk_norm_rope_backward(None, k, None, cu[1], None, c["rule"], q_offset=c["cu"]["off"], grad_dtype=F32)
    x = c["x"].split([Hq, Hkv, Hkv], dim=2)
    for got, rows, w, g in ((both[3], x[0], c["wq"], dy[0]), (both[4], x[1], c["wk"], dy[1]), (only_k[4], x[1], c["wk"], dy[1])):
        _, want, _, terms = ref.backward(rows, g.transpose(1, 2), w, c["eps"], c["pos"], c["f"], inter)
        # sums run in chains of at most a warp's rows (48), the CTA's slots (64) and the grid's CTAs (10 a thread, then 5 steps)
        assert ((got.double().cpu() - want).abs() <= (48 + 64 + 16 + 64) * ref.U32 * terms).all()
