"""What the binding hands to kernels that write it (workspace, status, counters) is checked for place, type and size first, and the C
entries of the 8-bit cache refuse misaligned arrays. No GPU is needed."""
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


def strided(n):
    return torch.zeros(2 * n, dtype=torch.uint8)[::2]


BAD_STATUS = [torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int64), torch.zeros(1, dtype=torch.int32, device="meta")]
BAD_COUNTERS = [torch.zeros(3, dtype=torch.int64), torch.zeros(4, dtype=torch.int32), torch.zeros(8, dtype=torch.int64)[::2],
                torch.zeros(4, dtype=torch.int64, device="meta")]
BAD_WORKSPACE = [strided(1 << 16), torch.zeros(1 << 16, dtype=torch.uint8, device="meta")]


def calls(fa):
    """The entries on tensors of the CPU, which they refuse last."""
    f8, bf = torch.float8_e4m3fn, torch.bfloat16
    pages = torch.zeros(2, 2, 64, 64, dtype=torch.uint8).view(f8)
    scales, table = torch.ones(2, 2, 2), torch.zeros(1, 2, dtype=torch.int32)
    cache = (pages, pages, scales, scales, table)
    rows = torch.zeros(1, 4, 2, 64, dtype=bf)
    grad = torch.zeros(1, 2, 4, 64)
    return (lambda **kw: fa.flex_decode_fp8(torch.zeros(1, 4, 64, dtype=bf), *cache, None, **kw),
            lambda **kw: fa.flex_forward_paged_fp8(torch.zeros(1, 4, 8, 64, dtype=bf), *cache, None, 128, **kw),
            lambda **kw: fa.qk_norm_rope_backward(rows, None, grad, None, None, fa.make_qk_rule(torch.ones(64)), **kw))


def test_scratch_is_checked(fa):
    decode, prefill, backward = calls(fa)
    for call in (decode, prefill):
        for bad in BAD_STATUS:
            with pytest.raises(ValueError, match="status"):
                call(status=bad)
    for bad in BAD_COUNTERS:
        with pytest.raises(ValueError, match="counters"):
            decode(counters=bad)
    for call in (decode, prefill, backward):
        for bad in BAD_WORKSPACE:
            with pytest.raises(ValueError, match="workspace"):
                call(workspace=bad)
        with pytest.raises(ValueError, match="CUDA"):  # all of these are fine: what is refused is the CPU
            call(workspace=torch.zeros(1 << 16, dtype=torch.uint8))
    assert fa._scratch(torch.zeros(3, 5), torch.device("cpu")) == 60 and fa._scratch(None, torch.device("cpu")) == 0


def test_misaligned_arrays_are_refused(fa):
    lib, ok = fa.load(), ctypes.c_void_p(4096)

    def mask(q_len, bq, bk):
        c = fa.BlockMaskC()
        c.Bm, c.Hm, c.q_len, c.kv_len, c.bq, c.bk = 1, 1, q_len, 256, bq, bk
        c.nq, c.nk = -(-q_len // bq), 256 // bk
        for name in ("kv_num", "kv_idx", "full_kv_num", "full_kv_idx", "q_num", "q_idx", "full_q_num", "full_q_idx", "block_class"):
            setattr(c, name, 4096)
        c.rule = fa.make_mask_rule([("causal",)])
        return ctypes.byref(c)

    one, many = mask(1, 1, 64), mask(64, 128, 128)

    def decode(ks=ok, vs=ok, table=ok, out=ok, kind=1, lse=ok, status=None, counters=None):
        return lib.fa_flex_decode_fp8(ok, ok, ok, ks, vs, table, 9, one, None, 0.0, out, kind, lse, 2, 4, 2, 64, 64, 4, ok, 1 << 30,
                                      status, counters, None)

    def prefill(ks=ok, vs=ok, table=ok, out=ok, lse=ok, status=None):
        return lib.fa_flex_forward_paged_fp8(ok, ok, ok, ks, vs, table, 9, 64, 4, many, None, 0.0, out, 1, lse, 1, 4, 2, 64, 256, 64, 0, ok,
                                             1 << 30, status, None)

    odd = ctypes.c_void_p(4098)
    for name in ("ks", "vs", "table", "out", "lse", "status"):
        assert decode(**{name: odd}) == fa.ERR_INVALID_ARG, name
        assert prefill(**{name: odd}) == fa.ERR_INVALID_ARG, name
    assert decode(out=ctypes.c_void_p(4097), kind=0) == fa.ERR_INVALID_ARG
    assert decode(counters=ctypes.c_void_p(4100)) == fa.ERR_INVALID_ARG

    row = fa.RowsC(4096, 4096, 512, 64)
    for fn, scales in ((lib.fa_kv_append, ()), (lib.fa_kv_append_fp8, (ok, ok))):
        assert fn(None, ctypes.byref(row), ctypes.byref(row), None, None, None, None, ok, ok, *scales, ok, 9, 64, 4, 2, 4, 2, 8, 64, odd,
                  None) == fa.ERR_INVALID_ARG


@pytest.mark.gpu
def test_scratch_of_another_device_is_refused_on_the_gpu(fa):
    bf, f8 = torch.bfloat16, torch.float8_e4m3fn
    pages = torch.zeros(2, 2, 64, 64, dtype=torch.uint8, device="cuda").view(f8)
    scales, table = torch.ones(2, 2, 2, device="cuda"), torch.zeros(1, 2, dtype=torch.int32, device="cuda")
    cache = (pages, pages, scales, scales, table)
    rule = fa.make_mask_rule([("causal",)])
    one, many = (fa.create_block_mask(rule, 1, 4, n, 128, bq, bk) for n, bq, bk in ((1, 1, 64), (8, 128, 128)))
    q1, q8 = torch.zeros(1, 4, 64, dtype=bf, device="cuda"), torch.zeros(1, 4, 8, 64, dtype=bf, device="cuda")
    for bad in (dict(status=torch.zeros(1, dtype=torch.int32)), dict(workspace=torch.zeros(1 << 20, dtype=torch.uint8)),
                dict(workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))):  # (the last: too small, found by the C entry)
        with pytest.raises((ValueError, RuntimeError)):
            fa.flex_decode_fp8(q1, *cache, one, **bad)
        with pytest.raises((ValueError, RuntimeError)):
            fa.flex_forward_paged_fp8(q8, *cache, many, 128, **bad)
    with pytest.raises(ValueError):
        fa.flex_decode_fp8(q1, *cache, one, counters=torch.zeros(4, dtype=torch.int64))
    # a workspace of another type is taken by its bytes
    n = fa.decode_fp8_workspace_bytes(1, 4, 2, 64, 2, 64)
    out = fa.flex_decode_fp8(q1, *cache, one, workspace=torch.zeros(-(-n // 4), device="cuda"))[0]
    assert not out.any()
