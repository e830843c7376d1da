"""Refusals of the key-block bounds and of the choice of blocks: argument errors come back as codes (or ValueError from the binding)
before anything is launched. No GPU is needed."""
import ctypes

import pytest
import torch

from block_sparse_masked_create_gb300 import build as fa_build


@pytest.fixture(scope="module")
def fa():
    fa_build.build()
    from block_sparse_masked_create_gb300 import fa as m
    m.load()
    return m


P = ctypes.c_void_p(4096)
OFF = ctypes.c_void_p(4104)   # misaligned for rows of 16 bytes
ODD = ctypes.c_void_p(4098)   # misaligned for 32-bit words


def test_key_bounds_refusals(fa):
    def call(k=P, out=P, B=2, Hkv=2, n=100, d=64, Bk=32):
        return fa.load().fa_key_bounds(k, out, B, Hkv, n, d, Bk, None)

    for bad in (dict(k=None), dict(out=None), dict(k=OFF), dict(out=OFF)):
        assert call(**bad) == fa.ERR_INVALID_ARG, bad
    for bad in (dict(B=0), dict(Hkv=0), dict(n=0), dict(Bk=0), dict(Bk=129), dict(Bk=-1)):
        assert call(**bad) == fa.ERR_SHAPE, bad
    for bad in (dict(d=96), dict(B=65536), dict(Hkv=65536)):
        assert call(**bad) == fa.ERR_UNSUPPORTED, bad


@pytest.mark.parametrize("fp8", [False, True])
def test_kv_bounds_refusals(fa, fp8):
    def call(k=P, ks=P, out=P, table=P, off=None, n_new=None, pages=8, page=64, max_pages=4, B=2, Hkv=2, N=3, d=64, status=None):
        tail = (out, table, off, n_new, pages, page, max_pages, B, Hkv, N, d, status, None)
        return fa.load().fa_kv_bounds_fp8(k, ks, *tail) if fp8 else fa.load().fa_kv_bounds(k, *tail)

    bads = [dict(k=None), dict(out=None), dict(table=None), dict(k=OFF), dict(out=OFF), dict(table=ODD), dict(off=ODD), dict(n_new=ODD), dict(status=ODD)]
    for bad in bads + ([dict(ks=None), dict(ks=ODD)] if fp8 else []):
        assert call(**bad) == fa.ERR_INVALID_ARG, bad
    for bad in (dict(B=0), dict(Hkv=0), dict(N=0), dict(pages=0), dict(max_pages=0)):
        assert call(**bad) == fa.ERR_SHAPE, bad
    for bad in (dict(d=32), dict(page=48), dict(page=256), dict(page=0), dict(B=65536)) + ((dict(page=16),) if fp8 else ()):
        assert call(**bad) == fa.ERR_UNSUPPORTED, bad


def mask(fa, nq=2, nk=4, bq=128, bk=64, q_len=256, kv_len=256, Bm=1, Hm=1):
    c = fa.BlockMaskC()
    c.Bm, c.Hm, c.q_len, c.kv_len, c.bq, c.bk, c.nq, c.nk = Bm, Hm, q_len, kv_len, bq, bk, nq, nk
    for name in ("kv_num", "kv_idx", "full_kv_num", "full_kv_idx", "q_num", "q_idx", "full_q_num", "full_q_idx", "block_class"):
        setattr(c, name, 4096)
    c.rule = fa.make_mask_rule([("causal",)])
    return c


def test_select_blocks_refusals(fa):
    lib = fa.load()
    big = ctypes.c_void_p(1 << 20)

    def call(c=0, q=P, box=P, table=None, pages=0, max_pages=0, B=2, Hq=4, Hkv=2, d=64, keep=3, first=1, last=1, buf=big, n=1 << 40, out=0, ws=big,
             wn=1 << 40, status=None):
        c = mask(fa) if c == 0 else c
        out = fa.BlockMaskC() if out == 0 else out
        return lib.fa_block_mask_select_blocks(ctypes.byref(c) if c else None, q, box, table, pages, max_pages, B, Hq, Hkv, d, keep, first, last, buf, n,
                                               ctypes.byref(out) if out else None, ws, wn, status, None)

    none = mask(fa)
    none.block_class = None
    bads = [dict(c=None), dict(q=None), dict(box=None), dict(buf=None), dict(out=None), dict(ws=None), dict(q=OFF), dict(box=OFF), dict(table=ODD, pages=8, max_pages=4),
            dict(status=ODD), dict(buf=P.value and ctypes.c_void_p((1 << 20) + 128)), dict(ws=ctypes.c_void_p((1 << 20) + 16)), dict(c=none),
            dict(keep=0), dict(keep=-1), dict(first=-1), dict(last=-1), dict(first=2, last=2), dict(first=2**31 - 1, last=2**31 - 1)]
    for bad in bads:
        assert call(**bad) == fa.ERR_INVALID_ARG, bad
    for bad in (dict(B=0), dict(Hq=0), dict(Hkv=0), dict(Hq=3), dict(c=mask(fa, Bm=3)), dict(c=mask(fa, nq=3)), dict(c=mask(fa, nk=3)), dict(c=mask(fa, bk=0)),
                dict(table=P, pages=0, max_pages=4), dict(table=P, pages=8, max_pages=3)):
        assert call(**bad) == fa.ERR_SHAPE, bad
    wide = mask(fa, nk=32769, bk=1, kv_len=32769)
    tall = mask(fa, nq=524281, bq=1, q_len=524281, nk=1, bk=128, kv_len=128)
    for bad in (dict(c=mask(fa, Hm=2)), dict(d=96), dict(c=wide), dict(c=tall), dict(B=65536), dict(Hq=65536, Hkv=65536)):
        assert call(**bad) == fa.ERR_UNSUPPORTED, bad
    c = mask(fa)
    n = lib.fa_block_mask_select_blocks_bytes(ctypes.byref(c), 2, 2)
    wn = lib.fa_block_mask_select_blocks_workspace_bytes(ctypes.byref(c), 2, 4, 2, 64)
    assert n >= 2 * 2 * 2 * 4 * 17 and wn >= 2 * 2 * 2 * 4 * 8
    assert call(n=n - 1) == fa.ERR_BUFFER and call(wn=wn - 1) == fa.ERR_BUFFER
    one = mask(fa, nq=1, bq=1, q_len=1)                                # one query: no workspace, unless its row is very long
    assert lib.fa_block_mask_select_blocks_workspace_bytes(ctypes.byref(one), 2, 4, 2, 64) == 0
    assert call(c=one, ws=None, wn=0, n=0) == fa.ERR_BUFFER
    one = mask(fa, nq=1, bq=1, q_len=1, nk=2049, bk=64, kv_len=2049 * 64)
    assert lib.fa_block_mask_select_blocks_workspace_bytes(ctypes.byref(one), 2, 4, 2, 64) >= 2 * 2 * 2049 * 8
    assert call(c=one, ws=None) == fa.ERR_INVALID_ARG
    assert lib.fa_block_mask_select_blocks_bytes(None, 2, 2) == 0
    assert lib.fa_block_mask_select_blocks_workspace_bytes(ctypes.byref(mask(fa)), 2, 3, 2, 64) == 0


def test_select_blocks_refuses_the_buffer_that_it_reads(fa):
    lib = fa.load()
    c = mask(fa)
    n = lib.fa_block_mask_select_blocks_bytes(ctypes.byref(c), 2, 2)
    out = fa.BlockMaskC()
    for at in (1 << 20, (1 << 20) + n - 1, (1 << 20) - c.Bm * c.nq * c.nk + 1):   # its first byte, its last, and classes that end on its first
        c.block_class = at
        assert lib.fa_block_mask_select_blocks(ctypes.byref(c), P, P, None, 0, 0, 2, 4, 2, 64, 3, 1, 1, ctypes.c_void_p(1 << 20), n, ctypes.byref(out),
                                               ctypes.c_void_p(1 << 30), 1 << 30, None, None) == fa.ERR_INVALID_ARG


def test_decode_takes_one_row_for_all_heads_or_one_for_each_kv_head(fa):
    lib = fa.load()
    for hm, code in ((3, fa.ERR_SHAPE), (8, fa.ERR_SHAPE), (2, fa.ERR_BUFFER), (1, fa.ERR_BUFFER)):
        c = mask(fa, nq=1, nk=4, bq=1, bk=64, q_len=1, kv_len=256, Hm=hm)
        assert lib.fa_flex_decode(P, P, P, P, 8, ctypes.byref(c), None, 0.0, P, 0, P, 1, 8, 2, 64, 64, 4, P, 0, None, None, None) == code, hm
        assert lib.fa_flex_decode_fp8(P, P, P, P, P, P, 8, ctypes.byref(c), None, 0.0, P, 0, P, 1, 8, 2, 64, 64, 4, P, 0, None, None, None) == code, hm


def test_forward_and_backward_refuse_other_head_counts(fa):
    lib = fa.load()
    c = mask(fa, Hm=4)
    assert lib.fa_flex_forward(P, P, P, ctypes.byref(c), None, 0.0, P, 0, P, 1, 8, 2, 256, 256, 64, None, None, None) == fa.ERR_SHAPE
    assert lib.fa_flex_backward(P, P, P, P, 0, P, P, ctypes.byref(c), None, 0.0, P, P, P, P, 1, 8, 2, 256, 256, 64, None, None) == fa.ERR_SHAPE


def test_binding_refuses_host_tensors(fa):
    x = torch.zeros(1, 2, 64, 64, dtype=torch.bfloat16)
    table = torch.zeros(1, 1, dtype=torch.int32)
    with pytest.raises(ValueError):
        fa.key_bounds(x)
    with pytest.raises(ValueError):
        fa.kv_bounds(x, x, table)
    with pytest.raises(ValueError):
        fa.kv_bounds_fp8(x, None, x, table)
    with pytest.raises(ValueError):
        fa.select_blocks(fa.BlockMask(fa.BlockMaskC(), x), x, x, 2)
