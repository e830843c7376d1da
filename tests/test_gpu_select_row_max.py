"""Decodes over a mask whose row_max is not what its rows list."""
import pytest
import torch

from gpu_common import LSE_MAX, O_MAX
from test_gpu_select import cache, fa, paged_case  # noqa: F401 (fa is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d,page,Hq,Hkv", [(128, 64, 8, 2), (64, 32, 4, 4), (128, 32, 4, 1)])
def test_rows_longer_than_the_mask_says(fa, fp8, d, page, Hq, Hkv):  # noqa: F811
    lens = [40 * page, 1, 2 * page]
    src, q, box, table, _ = paged_case(fa, 3, lens, Hq, Hkv, d, page, 5)
    (k, ks), (v, vs) = cache(box.shape[0], Hkv, page, d, 6, fp8), cache(box.shape[0], Hkv, page, d, 7, fp8)
    bm = fa.select_blocks(src, q, box, 30, 1, 1, page_table=table)
    q = q[:, :, 0].contiguous()

    def decode(most):
        bm.c.row_max = most
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        size = fa.decode_fp8_workspace_bytes(3, Hq, Hkv, d, table.shape[1], page) if fp8 else fa.decode_workspace_bytes(3, Hq, d, table.shape[1], page)
        ws = torch.full((size,), 0x7F, dtype=torch.uint8, device="cuda")       # NaN where nothing was written
        args = (k, v, ks, vs, table, bm) if fp8 else (k, v, table, bm)
        run = fa.flex_decode_fp8 if fp8 else fa.flex_decode
        o, lse = run(q, *args, workspace=ws, status=status, out_dtype=torch.float32)
        return fa.check_status(status), o, lse

    st, o, lse = decode(30)
    assert st == fa.OK
    far = 2 * O_MAX * max(1.0, float(o.abs().max()))       # each result lies within O_MAX (of values of magnitude 1) of the 64-bit one
    for most in (0, -1, 40, 2**31 - 1):            # not known, or more than there are: the same result but for the order of the sums
        st, o2, lse2 = decode(most)
        assert st == fa.OK and torch.allclose(o, o2, atol=far, rtol=0) and torch.allclose(lse, lse2, atol=2 * LSE_MAX, rtol=0)
    for most in (1, 2, 7):
        st, o2, lse2 = decode(most)
        assert st == fa.ERR_DEVICE_CHECK
        assert bool(o2.isfinite().all()) and bool(lse2.isfinite().all())
        assert torch.allclose(o[1], o2[1], atol=far, rtol=0) and torch.allclose(lse[1], lse2[1], atol=2 * LSE_MAX, rtol=0)   # its row lists one block
