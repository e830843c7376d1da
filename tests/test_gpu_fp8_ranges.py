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


# ------------------------------------------------------------------------------------------ V scales far apart
@pytest.mark.parametrize("factor", [2.0 ** 20, 2.0 ** 30, 2.0 ** 45])
@pytest.mark.parametrize("d,page,Q,Hq", [(128, 64, 150, 4), (64, 32, 150, 4), (64, 128, 30, 6)])
def test_prefill_large_v_scale_that_a_row_does_not_see(factor, d, page, Q, Hq):
    # tokens 256 .. 287 are seen by the first rows of Q = 150 and by none of Q = 30
    L, window = 390, 40
    cached = cache(62, [L], 2, page, d)
    cached[3][cached[4][0, 256 // page], :, 256 % page // 32] *= factor
    q = torch.randn(1, Hq, Q, d, generator=gen(63)).to(BF)
    i, j = L - Q + torch.arange(Q)[:, None], torch.arange(L)[None]
    al = (j <= i) & (i - j < window)
    want = request(q, cached, 0, L, i, al)
    # a key's share in units of at most 2 times the row's largest
    want = widened(want, subnormal_floor(q, cached, 0, L, al, d ** -0.5, 2.0, of_block=False))
    for chunk in (-1, 1):
        out, lse, st = forward(q, cached, [L], [L - Q], window, chunk=chunk)
        assert st == fa.OK
        close(out[0], lse[0], want, d, 0.0, F32, 2.0 ** -18, f"chunk {chunk}")


@pytest.mark.parametrize("bk,Q,Hq,Hkv,d", [(128, 90, 8, 2, 64), (128, 20, 6, 2, 128), (64, 90, 8, 2, 64), (128, 150, 16, 1, 64)])
def test_prefill_of_a_padded_batch_over_a_used_pool(bk, Q, Hq, Hkv, d):
    # prompts of several lengths appended and attended in one call each: rows behind a prompt see what the pool held before (bytes
    # without NaN, any scales), and the prompt's rows are right all the same
    B, page = 3, 64
    lens = [Q, Q // 3, Q - 7]
    g = gen(66)
    each = -(-Q // page)
    table = torch.randperm(B * each + 1, generator=g)[:B * each].view(B, each).to(torch.int32)

    def pool():
        x = torch.randint(0, 256, (B * each + 1, Hkv, page, d), generator=g, dtype=torch.uint8)
        x[(x & 0x7F) == NAN_BYTE] = 0
        s = torch.tensor([2.0 ** 60, math.inf, math.nan, 0.0, -1.0, 2.0 ** 38])[torch.randint(0, 6, (B * each + 1, Hkv, page // 32), generator=g)]
        return x.cuda().view(F8), s.cuda()

    (kp, ks), (vp, vs) = pool(), pool()
    x = torch.randn(B, Q, Hq + 2 * Hkv, d, generator=g).to(BF).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = fa.kv_append_fp8(*x.split([Hq, Hkv, Hkv], dim=2), kp, vp, ks, vs, table.cuda(), n_new=torch.tensor(lens, dtype=torch.int32).cuda(), status=status)
    assert fa.check_status(status) == fa.OK
    q = q.cpu()
    for b, L in enumerate(lens):
        q[b, :, L:] = 1.0  # rows that the append leaves as they are
    cached = tuple(t.cpu() for t in (kp, vp, ks, vs)) + (table,)
    out, lse, st = forward(q, cached, lens, [0] * B, bk=bk, n=Q)
    assert st == fa.OK
    for b, L in enumerate(lens):
        i, j = torch.arange(L)[:, None], torch.arange(L)[None]
        want = request(q[:, :, :L], cached, b, L, i, j <= i)
        if bk == 128 and -(-Q // 128) * (Hq // Hkv) <= 16:
            close(out[b, :, :L], lse[b, :, :L], want, d, 0.0, F32, 0.0, f"request {b}")
        else:  # expanded: P is bf16
            assert ((out[b, :, :L].double().cpu() - want[0]).abs() <= (2.0 ** -8 + 2.0 ** -10) * want[2] + 1e-4).all()
            assert (lse[b, :, :L].double().cpu() - want[1]).abs().max() <= 2e-3


# ------------------------------------------------------------------------------------------ one key outweighs a long row
def sink_case(L, at, d, Hkv):
    """Keys of zero but for token `at`, which q = (4, 0 ..) scores 128 * scale; V is 1 but for that token's, which is 0."""
    page = 64
    kp, vp, ks, vs, table = cache(67, [L], Hkv, page, d)
    kp.zero_()
    vp.copy_(torch.full_like(vp, 256.0, dtype=F32).to(F8))
    ks.fill_(2.0 ** -40)
    vs.fill_(2.0 ** -8)
    kp[table[0, at // page], :, at % page, 0] = 256.0
    ks[table[0, at // page], :, at % page // 32] = 2.0 ** -3
    vp[table[0, at // page], :, at % page] = 0.0
    return kp, vp, ks, vs, table


@pytest.mark.parametrize("lead", [10.0, 14.0, 17.0, 17.4, 20.0, 26.0])
@pytest.mark.parametrize("Q,Hq,d,at", [(130, 1, 64, 0), (130, 1, 64, 9999), (30, 4, 128, 0), (1, 2, 64, 40)])
def test_prefill_one_key_outweighs_a_long_row(lead, Q, Hq, d, at):
    L = 20000
    cached = sink_case(L, at, d, 1)
    q = torch.zeros(1, Hq, Q, d)
    q[..., 0] = 4.0
    q, scale = q.to(BF), lead / 128
    i, j = L - Q + torch.arange(Q)[:, None], torch.arange(L)[None]
    want = request(q, cached, 0, L, i, j <= i, scale)
    # units of at most twice a block's largest share
    want = widened(want, subnormal_floor(q, cached, 0, L, j <= i, scale, 2.0 ** -7 if at == 0 else 2.0))
    for chunk in (-1, 0, 5):
        out, lse, st = forward(q, cached, [L], [L - Q], chunk=chunk, scale=scale)
        assert st == fa.OK
        close(out[0], lse[0], want, d, 0.0, F32, 2.0 ** -18, f"chunk {chunk}")


def test_prefill_scores_that_fall_and_rise():
    # scores that fall by 60 and rise by 100 (base 2) over the row, V scales that go the other way: the reference follows
    L, Q, d, page = 2000, 130, 64, 64
    kp, vp, ks, vs, table = cache(68, [L], 1, page, d)
    t = torch.arange(L // 32 + 2).float()
    level = torch.where(t < 25, -2.0 * t, -50 + 2.5 * (t - 25)).round()
    kp.zero_()
    kp[..., 0] = torch.full(kp[..., 0].shape, 256.0).to(F8)
    for c in range(-(-L // 32)):
        p, s = int(table[0, c * 32 // page]), c * 32 % page // 32
        kp[p, 0, s * 32:s * 32 + 32, 0] = torch.tensor(float(level[c])).to(F8)
        ks[p, 0, s] = 1.0
        vs[p, 0, s] = 2.0 ** float(-level[c] / 2).__round__()
    q = torch.zeros(1, 2, Q, d)
    q[..., 0] = 1.0
    q, cached = q.to(BF), (kp, vp, ks, vs, table)
    i, j = L - Q + torch.arange(Q)[:, None], torch.arange(L)[None]
    want = widened(request(q, cached, 0, L, i, j <= i, 0.7), subnormal_floor(q, cached, 0, L, j <= i, 0.7, 2.0))
    for chunk in (-1, 3):
        out, lse, st = forward(q, cached, [L], [L - Q], chunk=chunk, scale=0.7)
        assert st == fa.OK
        close(out[0], lse[0], want, d, 0.0, F32, 2.0 ** -18, f"chunk {chunk}")


@pytest.mark.parametrize("power", [True, False])
@pytest.mark.parametrize("d,page,Q,Hq", [(128, 64, 150, 4), (64, 128, 30, 6)])
def test_prefill_v_scales_2_to_the_30_apart(power, d, page, Q, Hq):
    lens = [150, 390]
    kp, _, ks, _, table = cache(64, lens, 2, page, d, power=power)
    _, vp, _, vs, _ = cache(64, lens, 2, page, d, 30, power=power)
    cached = kp, vp, ks, vs, table
    q = torch.randn(2, Hq, Q, d, generator=gen(65)).to(BF)
    off = [L - Q for L in lens]
    for chunk in (-1, 1):
        out, lse, st = forward(q, cached, lens, off, chunk=chunk)
        assert st == fa.OK
        for b, L in enumerate(lens):
            i, j = off[b] + torch.arange(Q)[:, None], torch.arange(L)[None]
            want = widened(request(q, cached, b, L, i, j <= i), subnormal_floor(q, cached, b, L, j <= i, d ** -0.5, 2.0))
            # the row sum is held in the unit of p * v_scale: a logarithm of up to 2^6 is added to the LSE (2^-19), and the logarithms
            # of scales that are no powers of two are good to 2^-19
            close(out[b], lse[b], want, d, 0.0, F32, 2.0 ** -18, f"request {b}, chunk {chunk}")


# ------------------------------------------------------------------------------------------ the same in the decode
@pytest.mark.parametrize("lead", [14.0, 17.4, 20.0])
@pytest.mark.parametrize("Hq,d,at", [(1, 64, 0), (4, 128, 5000), (16, 64, 0)])
def test_decode_one_key_outweighs_a_long_row(lead, Hq, d, at):
    L, page = 20000, 64
    cached = sink_case(L, at, d, 1)
    q = torch.zeros(1, Hq, d)
    q[..., 0] = 4.0
    q, scale = q.to(BF), lead / 128
    off = torch.tensor([L - 1], dtype=torch.int32).cuda()
    n = cached[4].shape[1] * page
    bm = fa.create_block_mask(fa.make_mask_rule([("causal",)], q_offset=off), 1, Hq, 1, n, 1, page, keep=[off])
    out, lse = fa.flex_decode_fp8(q.cuda(), *[t.cuda() for t in cached], bm, None, scale, out_dtype=F32)
    i, j = torch.tensor([[L - 1]]), torch.arange(L)[None]
    o, z, av, qk = request(q[:, :, None], cached, 0, L, i, j <= i, scale)
    # 2^-32 of the key's weight, which is under 1, for the 1024 keys at most that share its sum (V is 1)
    close(out[0][:, None], lse[0][:, None], (o, z, av + 1024 * 2.0 ** -32 * 2.0 ** 11, qk), d, 0.0, F32, 0.0, "decode")


# ------------------------------------------------------------------------------------------ hidden slots
@pytest.mark.parametrize("bk,page,Q,Hq,Hkv,d", [(128, 32, 30, 2, 2, 64), (128, 64, 30, 8, 2, 128), (64, 32, 30, 2, 1, 64), (128, 32, 140, 2, 2, 64),
                                                (128, 64, 140, 16, 1, 64)])
def test_prefill_slots_before_the_window_may_hold_anything(bk, page, Q, Hq, Hkv, d):
    # pages that fell out of every row's window are handed on: their table entries are gone, slots of the page where the window
    # begins hold NaN, scales too
    L, window = 390, 5
    cached = cache(69, [L], Hkv, page, d)
    q = torch.randn(1, Hq, Q, d, generator=gen(70)).to(BF)
    i, j = L - Q + torch.arange(Q)[:, None], torch.arange(L)[None]
    al = (j <= i) & (i - j < window)
    want = request(q, cached, 0, L, i, al)
    first = L - Q - window + 1
    kp, vp, ks, vs, table = cached
    for c in range(-(-L // page)):
        pid = int(table[0, c])
        for p, s in ((kp, ks), (vp, vs)):
            p.view(torch.uint8)[pid, :, :max(0, min(page, first - c * page))] = NAN_BYTE
            s[pid, :, :max(0, min(page, first - c * page)) // 32] = math.nan
        if (c + 1) * page <= first:
            table[0, c] = -1
    for chunk in (-1, 1) if bk == 128 else (-1,):
        out, lse, st = forward(q, cached, [L], [L - Q], window, bk=bk, chunk=chunk)
        assert st == fa.OK
        if bk == 128 and -(-Q // 128) * (Hq // Hkv) <= 16:
            close(out[0], lse[0], want, d, 0.0, F32, 2.0 ** -18, f"chunk {chunk}")
        else:
            assert ((out[0].double().cpu() - want[0]).abs() <= (2.0 ** -8 + 2.0 ** -10) * want[2] + 1e-4).all()
            assert (lse[0].double().cpu() - want[1]).abs().max() <= 2e-3


def test_prefill_window_and_prefix_keep_the_prefix():
    # a prefix term shows the first keys to every row: nothing is cut off before it
    L, Q, d = 390, 30, 64
    cached = cache(71, [L], 2, 32, d)
    q = torch.randn(1, 4, Q, d, generator=gen(72)).to(BF)
    i, j = L - Q + torch.arange(Q)[:, None], torch.arange(L)[None]
    _, al = spec_and_mask(5, 3, i, j)
    out, lse, st = forward(q, cached, [L], [L - Q], 5, prefix=3)
    assert st == fa.OK
    close(out[0], lse[0], request(q, cached, 0, L, i, al), d, 0.0, F32, 0.0, "prefix")


@pytest.mark.parametrize("bk,Hq,Hkv", [(128, 4, 2), (128, 2, 2), (64, 4, 2)])
def test_prefill_of_a_batch_padded_in_front(bk, Hq, Hkv):
    # rows at negative positions see nothing
    lens, Q, d = [40, 200, 1], 100, 64
    cached = cache(73, lens, Hkv, 64, d)
    q = torch.randn(3, Hq, Q, d, generator=gen(74)).to(BF)
    off = [L - Q for L in lens]
    out, lse, st = forward(q, cached, lens, off, bk=bk)
    assert st == fa.OK
    for b, L in enumerate(lens):
        i, j = off[b] + torch.arange(Q)[:, None], torch.arange(L)[None]
        want = request(q, cached, b, L, i, j <= i)
        pad = max(0, -off[b])
        assert not out[b, :, :pad].any() and lse[b, :, :pad].isneginf().all()
        if bk == 128:
            close(out[b], lse[b], want, d, 0.0, F32, 0.0, f"request {b}")
        else:
            assert ((out[b].double().cpu() - want[0]).abs() <= (2.0 ** -8 + 2.0 ** -10) * want[2] + 1e-4).all()


# ------------------------------------------------------------------------------------------ captured calls
@pytest.mark.parametrize("bk,Q,Hq,Hkv,d,chunk", [(128, 150, 4, 2, 128, 0), (128, 20, 6, 2, 64, 0), (128, 150, 4, 2, 64, 1), (64, 70, 4, 2, 64, -1),
                                                 (128, 150, 16, 1, 64, 2)])
def test_prefill_captured_twice_and_replayed_at_once(bk, Q, Hq, Hkv, d, chunk):
    # two graphs on two streams, each with a workspace of its own, replayed on inputs written after the capture
    L = 3000
    kp, vp, ks, vs, table = cache(77, [L], Hkv, 64, d)
    table = table.cuda()
    off = torch.tensor([L - Q], dtype=torch.int32).cuda()
    bm = fa.create_block_mask(fa.make_mask_rule([("causal",)], q_offset=off), 1, Hq, Q, L, bk, bk, keep=[off])
    need = max(fa.forward_paged_fp8_workspace_bytes(bm, 1, Hq, Hkv, d, chunk), 256)
    runs = []
    for i in range(2):
        hold = [torch.zeros_like(t, device="cuda") for t in (torch.zeros(1, Hq, Q, d, dtype=BF), kp, vp, ks, vs)]
        out, lse = torch.empty(1, Hq, Q, d, device="cuda"), torch.empty(1, Hq, Q, device="cuda")
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            call = lambda: fa.flex_forward_paged_fp8(*hold, table, bm, L, chunk_blocks=chunk, out=out, lse=lse, workspace=ws)  # noqa: B023,E731
            call()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                call()
        runs.append((s, graph, hold, out, lse, ws))
    torch.cuda.synchronize()
    want = []
    for i, (_, _, hold, _, _, _) in enumerate(runs):
        for t, x in zip(hold, (torch.randn(1, Hq, Q, d, generator=gen(79 + i)).to(BF), kp, vp, ks, vs * 2.0 ** i)):
            t.copy_(x)
        want.append(fa.flex_forward_paged_fp8(*hold, table, bm, L, chunk_blocks=chunk, out_dtype=F32))
    torch.cuda.synchronize()
    for _ in range(5):
        for s, graph, _, _, _, _ in runs:
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for (_, _, _, out, lse, _), (o, z) in zip(runs, want):
        assert torch.isfinite(o).all() and torch.equal(out, o) and torch.equal(lse, z)
