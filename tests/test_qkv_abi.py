"""Refusals of the operators around the attention's inputs and the 8-bit cache: argument errors come back as codes (or
ValueError from the binding) before anything is launched. No GPU is needed."""
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


def rows(fa, ptr=4096, sb=4096, sn=512, sh=64):
    return fa.RowsC(ptr, sb, sn, sh)


def rule(fa, **kw):
    r = fa.QkRule()
    r.q_weight, r.k_weight, r.eps, r.inv_freq, r.rot_dim, r.interleaved = 4096, 4096, 1e-6, 4096, 64, 0
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def ref(s):
    return None if s is None else ctypes.byref(s)


def test_norm_rope_refusals(fa):
    lib = fa.load()

    def call(q=0, r=0, out=P, off=None, B=2, Hq=4, Hkv=2, N=8, d=64):
        q = rows(fa) if q == 0 else q
        r = rule(fa) if r == 0 else r
        return lib.fa_qk_norm_rope(ref(q), None, None, ref(r), off, out, None, None, B, Hq, Hkv, N, d, None)

    assert call(r=None) == fa.ERR_INVALID_ARG
    assert call(q=None) == fa.ERR_INVALID_ARG                                # no rows at all
    assert call(out=None) == fa.ERR_INVALID_ARG
    assert call(out=ctypes.c_void_p(4098)) == fa.ERR_INVALID_ARG
    assert call(q=rows(fa, ptr=4104)) == fa.ERR_INVALID_ARG                  # alignment
    assert call(q=rows(fa, sn=516)) == fa.ERR_INVALID_ARG                    # stride
    assert call(off=ctypes.c_void_p(4098)) == fa.ERR_INVALID_ARG
    for bad in (dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(interleaved=2), dict(q_weight=4098)):
        assert call(r=rule(fa, **bad)) == fa.ERR_INVALID_ARG, bad
    for rot in (0, 8, 24, 80, -16):
        assert call(r=rule(fa, rot_dim=rot)) == fa.ERR_UNSUPPORTED, rot
    assert call(d=96) == fa.ERR_UNSUPPORTED
    assert call(Hq=3) == fa.ERR_SHAPE and call(N=0) == fa.ERR_SHAPE and call(B=0) == fa.ERR_SHAPE
    assert call(B=1 << 16, N=1 << 16) == fa.ERR_SHAPE


def test_norm_rope_backward_refusals(fa):
    lib = fa.load()
    n = lib.fa_qk_norm_rope_backward_workspace_bytes(2, 8, 64)
    assert n > 0 and lib.fa_qk_norm_rope_backward_workspace_bytes(0, 8, 64) == 0

    def call(q=0, dq=P, out=0, r=0, kind=0, dw=P, ws=P, nbytes=n, d=64):
        q = rows(fa) if q == 0 else q
        out = rows(fa) if out == 0 else out
        r = rule(fa) if r == 0 else r
        return lib.fa_qk_norm_rope_backward(ref(q), None, dq, None, None, ref(r), None, ref(out), None, None, kind, dw, None,
                                            2, 4, 2, 8, d, ws, nbytes, None)

    assert call(dq=None) == fa.ERR_INVALID_ARG
    assert call(r=None) == fa.ERR_INVALID_ARG
    assert call(q=None) == fa.ERR_INVALID_ARG                                # a norm needs its rows
    assert call(out=None) == fa.ERR_INVALID_ARG
    assert call(dw=None) == fa.ERR_INVALID_ARG
    assert call(ws=None) == fa.ERR_INVALID_ARG
    assert call(nbytes=n - 1) == fa.ERR_BUFFER
    assert call(kind=2) == fa.ERR_INVALID_ARG
    assert call(dq=ctypes.c_void_p(4100)) == fa.ERR_INVALID_ARG
    assert call(d=32) == fa.ERR_UNSUPPORTED


def test_append_refusals(fa):
    lib = fa.load()

    def call(k=0, v=0, q=None, qo=None, pages=P, scales=(P, P), table=P, total=9, page=64, max_pages=4, fp8=True, d=64, n_new=None):
        k = rows(fa) if k == 0 else k
        v = rows(fa) if v == 0 else v
        fn = lib.fa_kv_append_fp8 if fp8 else lib.fa_kv_append
        mid = scales if fp8 else ()
        return fn(ref(q), ref(k), ref(v), None, None, n_new, qo, pages, pages, *mid, table, total, page, max_pages, 2, 4, 2, 8, d, None,
                  None)

    for fp8 in (True, False):
        assert call(k=None, fp8=fp8) == fa.ERR_INVALID_ARG
        assert call(v=None, fp8=fp8) == fa.ERR_INVALID_ARG
        assert call(q=rows(fa), fp8=fp8) == fa.ERR_INVALID_ARG               # no q_out
        assert call(pages=None, fp8=fp8) == fa.ERR_INVALID_ARG
        assert call(pages=ctypes.c_void_p(4104), fp8=fp8) == fa.ERR_INVALID_ARG
        assert call(table=None, fp8=fp8) == fa.ERR_INVALID_ARG
        assert call(table=ctypes.c_void_p(4097), fp8=fp8) == fa.ERR_INVALID_ARG
        assert call(n_new=ctypes.c_void_p(4097), fp8=fp8) == fa.ERR_INVALID_ARG
        assert call(total=0, fp8=fp8) == fa.ERR_SHAPE and call(max_pages=0, fp8=fp8) == fa.ERR_SHAPE
        assert call(page=48, fp8=fp8) == fa.ERR_UNSUPPORTED and call(d=80, fp8=fp8) == fa.ERR_UNSUPPORTED
    assert call(page=16) == fa.ERR_UNSUPPORTED                               # shorter than a scale's block
    assert call(scales=(P, None)) == fa.ERR_INVALID_ARG


def mask(fa, q_len, kv_len, bq, bk):
    c = fa.BlockMaskC()
    c.Bm, c.Hm, c.q_len, c.kv_len, c.bq, c.bk = 1, 1, q_len, kv_len, bq, bk
    c.nq, c.nk = -(-q_len // bq), -(-kv_len // bk)
    for name in ("kv_num", "kv_idx", "full_kv_num", "full_kv_idx", "q_num", "q_idx", "full_q_num", "full_q_idx", "block_class"):
        setattr(c, name, 4096)
    c.rule = fa.make_mask_rule([("causal",)])
    return c


def test_decode_refusals(fa):
    lib = fa.load()
    c = mask(fa, 1, 256, 1, 64)
    n = lib.fa_decode_fp8_workspace_bytes(2, 4, 2, 64, 4, 64)
    assert n > 0 and lib.fa_decode_fp8_workspace_bytes(2, 4, 2, 64, 4, 16) == 0

    def call(q=P, s=P, kind=0, Hq=4, Hkv=2, d=64, page=64, max_pages=4, total=9, ws=P, nbytes=n, m=c):
        return lib.fa_flex_decode_fp8(q, P, P, s, s, P, total, ref(m), None, 0.0, P, kind, P, 2, Hq, Hkv, d, page, max_pages, ws, nbytes,
                                      None, None, None)

    assert call(q=None) == fa.ERR_INVALID_ARG and call(s=None) == fa.ERR_INVALID_ARG and call(ws=None) == fa.ERR_INVALID_ARG
    assert call(q=ctypes.c_void_p(4098)) == fa.ERR_INVALID_ARG and call(kind=3) == fa.ERR_INVALID_ARG
    assert call(Hq=5) == fa.ERR_SHAPE and call(total=0) == fa.ERR_SHAPE and call(max_pages=5) == fa.ERR_SHAPE
    assert call(d=96) == fa.ERR_UNSUPPORTED and call(page=16) == fa.ERR_UNSUPPORTED and call(Hq=34) == fa.ERR_UNSUPPORTED
    assert call(total=1 << 25) == fa.ERR_UNSUPPORTED                         # more rows than a copy's coordinate
    assert call(nbytes=n - 1) == fa.ERR_BUFFER
    assert call(m=mask(fa, 256, 256, 64, 64)) == fa.ERR_SHAPE                # a prefill mask


def test_prefill_refusals(fa):
    lib = fa.load()
    c = mask(fa, 64, 256, 128, 128)
    n = lib.fa_forward_paged_fp8_workspace_bytes(ref(c), None, 1, 4, 2, 64, 0)
    assert n > 0 and lib.fa_forward_paged_fp8_workspace_bytes(ref(c), None, 1, 4, 2, 64, -2) == 0

    def call(s=P, table=P, page=64, max_pages=4, total=9, Q=64, KV=256, chunk=0, ws=P, nbytes=n, m=c, d=64, kind=0):
        return lib.fa_flex_forward_paged_fp8(P, P, P, s, s, table, total, page, max_pages, ref(m), None, 0.0, P, kind, P, 1, 4, 2, Q, KV, d,
                                             chunk, ws, nbytes, None, None)

    assert call(s=None) == fa.ERR_INVALID_ARG and call(table=None) == fa.ERR_INVALID_ARG and call(ws=None) == fa.ERR_INVALID_ARG
    assert call(ws=ctypes.c_void_p(4112)) == fa.ERR_INVALID_ARG and call(kind=9) == fa.ERR_INVALID_ARG
    assert call(chunk=-2) == fa.ERR_INVALID_ARG
    assert call(page=48) == fa.ERR_UNSUPPORTED and call(d=80) == fa.ERR_UNSUPPORTED
    assert call(max_pages=3) == fa.ERR_SHAPE and call(total=0) == fa.ERR_SHAPE and call(KV=255) == fa.ERR_SHAPE
    assert call(nbytes=n - 1) == fa.ERR_BUFFER
    small = mask(fa, 64, 256, 64, 64)
    assert call(m=small, chunk=4, nbytes=1 << 40) == fa.ERR_UNSUPPORTED      # cut rows want 128 x 128 blocks
    assert call(m=mask(fa, 64, 256, 16, 16), nbytes=1 << 40) == fa.ERR_UNSUPPORTED
    small.q_num = None
    assert call(m=small, nbytes=1 << 40) == fa.ERR_INVALID_ARG               # no query-side transpose
    assert call(total=1 << 26) == fa.ERR_UNSUPPORTED                         # more rows than a copy's coordinate


def test_binding_checks_types_shapes_and_devices(fa):
    x = torch.zeros(1, 4, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fa.qk_norm_rope(x, None, None, fa.make_qk_rule())                    # on the CPU
    with pytest.raises(ValueError):
        fa.qk_norm_rope(None, None, None, fa.make_qk_rule())
    with pytest.raises(ValueError):
        fa.make_qk_rule(q_weight=torch.zeros(64, dtype=torch.float64))
    with pytest.raises(ValueError):
        fa.kv_append(None, None, x, x, x, torch.zeros(1, 1, dtype=torch.int32))
    with pytest.raises(ValueError):
        fa.kv_append_fp8(None, x, x, x, x, None, None, torch.zeros(1, 1, dtype=torch.int32))
    with pytest.raises(ValueError):
        fa.flex_decode_fp8(x[0], x, x, x, x, x, None)
