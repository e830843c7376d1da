"""Attention over the 8-bit paged cache on the GPU where the numbers or the masks are far from ordinary: queries near zero, V scales
far apart, one key that outweighs a long row, hidden slots that nobody wrote, padded batches, masks per head."""
import math

import pytest
import torch

from block_sparse_masked_create_gb300 import fa
from tests import qkv_ref as ref
from tests.test_gpu_fp8 import BF, F32, F8, NAN_BYTE, cache, close, gen, spec_and_mask

pytestmark = pytest.mark.gpu


def forward(q, cached, lens, off, window=0, bk=128, chunk=-1, n=None, scale=None, out_dtype=F32, head_dependent=False, prefix=0):
    """(out, lse, status) of the causal (windowed) forward over `cached` = (k pages, v pages, k scales, v scales, table)."""
    B, Hq, Q, d = q.shape
    n = n or max(lens)
    spec, _ = spec_and_mask(window, prefix, torch.zeros(1, 1), torch.zeros(1, 1))
    off_c = torch.tensor(off, dtype=torch.int32).cuda()
    bm = fa.create_block_mask(fa.make_mask_rule(spec, q_offset=off_c, head_dependent=head_dependent), B, Hq, Q, n, bk, bk, keep=[off_c])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = fa.flex_forward_paged_fp8(q.cuda(), *[t.cuda() for t in cached], bm, n, None, scale, chunk_blocks=chunk, status=status,
                                         out_dtype=out_dtype)
    return out, lse, fa.check_status(status)


def request(q, cached, b, L, i, al, scale=None):
    """ref.attention of one request's rows at positions i [Q, 1]."""
    kp, vp, ks, vs, table = cached
    dk, dv = ref.dequant(kp, ks), ref.dequant(vp, vs)
    return ref.attention(q[b].double(), ref.gather(dk, table[b], L), ref.gather(dv, table[b], L), al, scale or q.shape[-1] ** -0.5, pos=i[:, 0])


def subnormal_floor(q, cached, b, L, al, scale, unit, of_block=True):
    """What rows can lose [Hq, Q, d] where a key's share of O is subnormal in fp16: each key is off by at most half of fp16's smallest
    step, 2^-25, in units of `unit` times the largest p * v_scale of its 128-key block (of_block) or of the row, times |v8|."""
    kp, vp, ks, vs, table = cached
    Hkv, page = kp.shape[1], kp.shape[2]
    k = ref.gather(ref.dequant(kp, ks), table[b], L)
    v8 = ref.gather(vp.float().double(), table[b], L).abs()
    s = ref.gather(vs.double().repeat_interleave(32, -1)[..., None], table[b], L)[..., 0]
    pad = -L % 128
    out = []
    for h in range(q.shape[1]):
        hk = h // (q.shape[1] // Hkv)
        x = (scale * q[b, h].double() @ k[hk].nan_to_num(0).T).masked_fill(~al, -math.inf)
        w = torch.softmax(x, -1).nan_to_num(0) * s[hk].nan_to_num(0)
        top = torch.nn.functional.pad(w, (0, pad)).view(w.shape[0], -1, 128).amax(-1)
        if not of_block:
            top = top.amax(-1, keepdim=True).expand_as(top)
        mass = torch.nn.functional.pad(v8[hk].nan_to_num(0), (0, 0, 0, pad)).view(-1, 128, v8.shape[-1]).sum(1)
        out.append(2.0 ** -25 * unit * top @ mass)
    return torch.stack(out)


def widened(want, floor):
    o, z, av, qk = want
    return o, z, av + floor * 2.0 ** 11, qk


# ------------------------------------------------------------------------------------------ queries near zero
@pytest.mark.parametrize("q_scale", [1e-32, 1e-33, 1e-36, 1e-39])
@pytest.mark.parametrize("d,page,Q", [(128, 64, 150), (64, 128, 30), (128, 32, 1)])
def test_prefill_queries_near_zero(q_scale, d, page, Q):
    # a row's factor times the scale of a key block that no row sees, or of keys that are all zero, underflows
    lens = [150, 390]
    cached = cache(60, lens, 2, page, d)
    cached[2][cached[4][1, 0], :, 0] = 2.0 ** -40
    q = (torch.randn(2, 4, Q, d, generator=gen(61)) * q_scale).to(BF)
    off = [L - Q for L in lens]
    for chunk in (-1, 1):
        out, lse, st = forward(q, cached, lens, off, chunk=chunk)
        assert st == fa.OK
        for b, L in enumerate(lens):
            i, j = off[b] + torch.arange(Q)[:, None], torch.arange(L)[None]
            close(out[b], lse[b], request(q, cached, b, L, i, j <= i), d, 0.0, F32, 2.0 ** -18 if chunk > 0 else 0.0, f"request {b}")
