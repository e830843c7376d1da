"""Source masks and buffers that the choice of blocks refuses. No GPU is needed."""
import ctypes

import pytest

from test_select_abi import P, fa, mask  # noqa: F401 (fa is a fixture)

BIG = ctypes.c_void_p(1 << 20)


def choose(fa, c, B=2, buf=BIG, n=1 << 40):  # noqa: F811
    out = fa.BlockMaskC()
    return fa.load().fa_block_mask_select_blocks(ctypes.byref(c), P, P, None, 0, 0, B, 4, 2, 64, 3, 1, 1, buf, n, ctypes.byref(out), BIG, 1 << 40, None, None)


@pytest.mark.parametrize("q_len,nq,bq", [(256, 2, 128), (1, 1, 1)])
def test_one_offset_for_several_batch_rows(fa, q_len, nq, bq):  # noqa: F811
    # the result would have a row set for each batch row and read an offset for each: there is one
    c = mask(fa, nq=nq, q_len=q_len, bq=bq)
    c.rule.q_offset = 4096
    for B in (2, 4, 65535):
        assert choose(fa, c, B) == fa.ERR_INVALID_ARG, B
    # one batch row, and an offset for each: the next check answers
    assert choose(fa, c, 1, n=0) == fa.ERR_BUFFER
    c = mask(fa, nq=nq, q_len=q_len, bq=bq, Bm=2)
    c.rule.q_offset = 4096
    assert choose(fa, c, 2, n=0) == fa.ERR_BUFFER


def test_more_heads_than_a_row_set_is_found_for(fa):  # noqa: F811
    # the row set of a query head is found by a product that is exact for Hq times the group's heads under 2^32
    lib = fa.load()
    c = mask(fa, Hm=2)
    for Hq, code in ((2**17, fa.ERR_UNSUPPORTED), (2**16, fa.ERR_INVALID_ARG)):
        assert lib.fa_flex_forward(P, P, P, ctypes.byref(c), None, 0.0, ctypes.c_void_p(4104), 0, P, 1, Hq, 2, 256, 256, 64, None, None, None) == code


def test_a_buffer_that_holds_the_document_runs(fa):  # noqa: F811
    # a choice keeps the runs of the mask that it was made from: a choice from it must not be laid out over them
    c = mask(fa)
    c.rule.doc_batch, c.rule.doc_len = 1, 256
    n = fa.load().fa_block_mask_select_blocks_bytes(ctypes.byref(c), 2, 2)
    at = BIG.value
    for name, size in (("doc_run", 2 * 256 * 4), ("doc_sorted", 4)):
        for start, code in ((at, fa.ERR_INVALID_ARG), (at + n - 4, fa.ERR_INVALID_ARG), (at - size + 4, fa.ERR_INVALID_ARG)):
            setattr(c, name, start)
            assert choose(fa, c, buf=BIG, n=n) == code, (name, start)
        setattr(c, name, None)
