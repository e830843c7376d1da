"""fa_qk_norm_rope, its gradient, and fa_kv_append / fa_kv_append_fp8 on the GPU against 64-bit forms (tests/qkv_ref.py):
head layouts, strides, odd lengths, far positions, partial and interleaved rotation, padded batches, pages that end
inside a block, sequences cut back and continued, bad pages and positions, streams and captured graphs."""
import numpy as np
import pytest
import torch

from block_sparse_masked_create_gb300 import fa
from tests import qkv_ref as ref

pytestmark = pytest.mark.gpu
BF, F32, F8 = torch.bfloat16, torch.float32, ref.F8


def gen(seed):
    return torch.Generator().manual_seed(seed)


def inv_freq(rot, theta=10000.0):
    return None if not rot else (theta ** (-2 * torch.arange(rot // 2, dtype=torch.float64) / rot)).to(F32)


def make(seed, B, N, Hq, Hkv, d, rot, norm, interleaved=False, offset=0, eps=1e-6):
    g = gen(seed)
    x = torch.randn(B, N, Hq + 2 * Hkv, d, generator=g) * (1 + 7 * (torch.rand(d, generator=g) > 0.9))
    x = x.to(BF)
    wq, wk = ((1 + 0.3 * torch.randn(d, generator=g)) if norm else None for _ in range(2))
    off = torch.randint(0, 50, (B,), generator=g).to(torch.int32) + offset
    c = dict(x=x, wq=wq, wk=wk, eps=eps, f=inv_freq(rot), inter=interleaved, off=off, B=B, N=N, Hq=Hq, Hkv=Hkv, d=d)
    c["pos"] = off.long()[:, None] + torch.arange(N)
    c["cu"] = {k: None if c[k] is None else c[k].cuda() for k in ("x", "wq", "wk", "f", "off")}
    c["rule"] = fa.make_qk_rule(c["cu"]["wq"], c["cu"]["wk"], eps, c["cu"]["f"], interleaved)
    return c


def split(c, x=None):
    return (c["cu"]["x"] if x is None else x).split([c["Hq"], c["Hkv"], c["Hkv"]], dim=2)


def expect(c):
    """[(fp64 rows, slack before the last rounding)] of q, k, v [B, N, H, d]."""
    out = []
    for x, w, kind in zip(c["x"].split([c["Hq"], c["Hkv"], c["Hkv"]], dim=2), (c["wq"], c["wk"], None), "qkv"):
        if kind == "v":
            out.append((x.double(), torch.zeros_like(x.double())))
        else:
            a = (w, c["eps"], c["pos"], c["f"], c["inter"])
            out.append((ref.forward(x, *a), ref.forward_slack(x, *a)))
    return out


def near(got, want, slack, dtype, what):
    err = (got.double().cpu() - want).abs()
    bound = ref.HALF[dtype] * (want.abs() + slack) + slack
    assert torch.isfinite(got.float()).all(), what
    assert (err <= bound).all(), f"{what}: {float((err - bound).max()):.3e} over the bound"


CASES = [  # B, N, Hq, Hkv, d, rot, norm, interleaved, offset
    (1, 1, 1, 1, 64, 64, True, False, 0),
    (2, 5, 4, 2, 128, 128, True, False, 0),
    (3, 67, 6, 2, 64, 32, True, True, 900001),
    (1, 130, 3, 3, 128, 48, False, False, 7),
    (2, 33, 8, 1, 128, 0, True, False, 0),
    (1, 9, 40, 8, 128, 112, True, True, 2 ** 31 - 100),
    (1, 300, 2, 1, 64, 16, False, True, 123456789),
]


@pytest.mark.parametrize("case", CASES)
def test_forward(case):
    c = make(1, *case[:6], case[6], case[7], case[8])
    outs = fa.qk_norm_rope(*split(c), c["rule"], q_offset=c["cu"]["off"])
    for o, (want, slack), kind in zip(outs, expect(c), "qkv"):
        near(o.transpose(1, 2), want, slack, BF, kind)
    assert torch.equal(outs[2].transpose(1, 2).cpu(), c["x"][:, :, c["Hq"] + c["Hkv"]:])


def test_forward_strides_and_left_out_rows():
    # the same rows as head-major tensors, as a slice of a wider tensor, and one kind at a time
    c = make(2, 2, 37, 4, 2, 128, 64, True)
    q, k, v = split(c)
    want = fa.qk_norm_rope(q, k, v, c["rule"], q_offset=c["cu"]["off"])
    hm = [t.transpose(1, 2).contiguous().transpose(1, 2) for t in (q, k, v)]
    wide = torch.full((2, 37, 8, 136), float("nan"), dtype=BF, device="cuda")
    wide[..., 8:] = c["cu"]["x"]
    for got in (fa.qk_norm_rope(*hm, c["rule"], q_offset=c["cu"]["off"]),
                fa.qk_norm_rope(*split(c, wide[..., 8:]), c["rule"], q_offset=c["cu"]["off"])):
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    for only in range(3):
        args = [t if i == only else None for i, t in enumerate((q, k, v))]
        got = fa.qk_norm_rope(*args, c["rule"], q_offset=c["cu"]["off"])
        for i in range(3):
            assert torch.equal(got[i], want[i]) if i == only else got[i] is None


def test_rows_of_zeros_infinities_and_nan_keep_to_themselves():
    c = make(3, 1, 8, 2, 1, 64, 64, True)
    x = c["cu"]["x"].clone()
    x[0, 1] = 0
    x[0, 3, 0, 5] = float("inf")
    x[0, 5, 2, 7] = float("nan")
    q, k, v = fa.qk_norm_rope(*split(c, x), c["rule"], q_offset=c["cu"]["off"])
    clean = fa.qk_norm_rope(*split(c), c["rule"], q_offset=c["cu"]["off"])
    assert not q[:, :, 1].any() and not k[:, :, 1].any()
    assert not torch.isfinite(q[0, 0, 3]).all() and torch.isnan(k[0, 0, 5]).any()
    for n in (0, 2, 4, 6, 7):
        for a, b in zip((q, k, v), clean):
            assert torch.equal(a[:, :, n], b[:, :, n])
    assert torch.equal(q[0, 1, 3], clean[0][0, 1, 3])


@pytest.mark.parametrize("inter", [False, True])
def test_an_infinity_stays_in_its_pair(inter):
    # no norm, a row rotated in part: an infinity reaches the other element of its own pair and nothing else
    c = make(31, 1, 4, 1, 1, 128, 32, False, inter, offset=3)
    clean = fa.qk_norm_rope(*split(c), c["rule"], q_offset=c["cu"]["off"])[0]
    for e, hit in ((77, {77}), (127, {127}), (34, {34}), (5, {4, 5} if inter else {5, 21})):
        x = c["cu"]["x"].clone()
        x[0, 2, 0, e] = float("inf")
        q = fa.qk_norm_rope(*split(c, x), c["rule"], q_offset=c["cu"]["off"])[0]
        other = [i for i in range(128) if i not in hit]
        assert torch.equal(q[..., other], clean[..., other]) and not torch.isfinite(q[0, 0, 2, e])
        g = torch.ones(1, 1, 4, 128, device="cuda")
        g[0, 0, 2, e] = float("inf")
        d = fa.qk_norm_rope_backward(None, None, g, None, None, c["rule"], q_offset=c["cu"]["off"])[0]
        assert torch.isfinite(d[..., other]).all() and not torch.isfinite(d[0, 2, 0, e])


# ------------------------------------------------------------------------------------------ gradient
@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_backward(case, dtype):
    c = make(4, *case[:6], case[6], case[7], case[8])
    g = gen(5)
    grads = [torch.randn(c["B"], h, c["N"], c["d"], generator=g) for h in (c["Hq"], c["Hkv"], c["Hkv"])]
    packed = torch.full(c["x"].shape, float("nan"), dtype=dtype, device="cuda")
    q, k, _ = split(c)
    a, b, v, dwq, dwk = fa.qk_norm_rope_backward(q, k, *[t.cuda() for t in grads], c["rule"], q_offset=c["cu"]["off"],
                                                 **dict(zip(("dq_in", "dk_in", "dv_in"), split(c, packed))))
    rows = c["x"].split([c["Hq"], c["Hkv"], c["Hkv"]], dim=2)
    for got, x, w, dy, dw, kind in ((a, rows[0], c["wq"], grads[0], dwq, "q"), (b, rows[1], c["wk"], grads[1], dwk, "k")):
        dx, want_w, slack, terms = ref.backward(x, dy.transpose(1, 2), w, c["eps"], c["pos"], c["f"], c["inter"])
        near(got, dx, slack, dtype, "d" + kind)
        assert (dw is None) == (w is None)
        if w is not None:  # at most one rounding a row, and those of a term
            n = c["B"] * c["N"] * x.shape[2]
            assert ((dw.double().cpu() - want_w).abs() <= (n + 64) * ref.U32 * terms).all(), kind
    near(v, grads[2].transpose(1, 2).double(), torch.zeros(1, dtype=torch.float64), dtype, "dv")


def test_backward_against_differences():
    # <dz, forward(x)> along a direction u, by a central difference of the 64-bit forward: its error is h^2 times the third
    # derivative (under 1e-6 of the sum of magnitudes for h = 1e-4) against fp32 gradients
    c = make(6, 2, 11, 3, 1, 64, 32, True)
    g = gen(7)
    dy = [torch.randn(2, h, 11, 64, generator=g) for h in (3, 1, 1)]
    q, k, _ = split(c)
    got = fa.qk_norm_rope_backward(q, k, *[t.cuda() for t in dy], c["rule"], q_offset=c["cu"]["off"], grad_dtype=F32)
    for x, w, d, dx, dw in ((c["x"][:, :, :3], c["wq"], dy[0], got[0], got[3]), (c["x"][:, :, 3:4], c["wk"], dy[1], got[1], got[4])):
        x, d = x.double(), d.transpose(1, 2).double()
        f = lambda xx, ww: (d * ref.rotate(xx * torch.rsqrt(xx.square().mean(-1, keepdim=True) + c["eps"]) * ww, c["pos"],
                                           c["f"], c["inter"])).sum()
        u, uw, h = torch.randn(x.shape, generator=g).double(), torch.randn(w.shape, generator=g).double(), 1e-4
        for diff, ana in (((f(x + h * u, w.double()) - f(x - h * u, w.double())) / (2 * h), dx.double().cpu() * u),
                          ((f(x, w.double() + h * uw) - f(x, w.double() - h * uw)) / (2 * h), dw.double().cpu() * uw)):
            assert abs(float(ana.sum() - diff)) <= 1e-5 * float(ana.abs().sum())


def test_backward_repeats_and_parts():
    c = make(8, 2, 700, 4, 2, 128, 128, True)
    g = gen(9)
    dy = [torch.randn(2, h, 700, 128, generator=g).cuda() for h in (4, 2, 2)]
    q, k, _ = split(c)
    one = fa.qk_norm_rope_backward(q, k, *dy, c["rule"], q_offset=c["cu"]["off"])
    two = fa.qk_norm_rope_backward(q, k, *dy, c["rule"], q_offset=c["cu"]["off"])
    for a, b in zip(one, two):
        assert torch.equal(a, b)
    only = fa.qk_norm_rope_backward(None, k, None, dy[1], None, c["rule"], q_offset=c["cu"]["off"])
    assert only[0] is None and only[2] is None and only[3] is None
    assert torch.equal(only[1], one[1])
    # another grid and another order of the heads inside a CTA: the weight's sum is rounded elsewhere
    assert (only[4] - one[4]).abs().max() <= 2 * (1400 * 2 + 64) * ref.U32 * one[4].abs().max() * 50


# ------------------------------------------------------------------------------------------ append
def tables(seed, B, pages_each, spare=2):
    g = gen(seed)
    total = B * pages_each + spare
    return torch.randperm(total, generator=g)[:B * pages_each].view(B, pages_each).to(torch.int32), total


@pytest.mark.parametrize("page,N,Hq,Hkv,d,rot,norm", [(16, 1, 4, 2, 64, 64, True), (32, 70, 4, 1, 128, 128, True),
                                                      (128, 1, 32, 8, 128, 128, True), (64, 5, 2, 2, 64, 0, False)])
def test_append_bf16(page, N, Hq, Hkv, d, rot, norm):
    B = 3
    c = make(10, B, N, Hq, Hkv, d, rot, norm)
    each = -(-(50 + N) // page)
    table, total = tables(11, B, each)
    n_new = torch.tensor([N, N // 2, 0], dtype=torch.int32)
    pools = [torch.randn(total, Hkv, page, d, generator=gen(12)).to(BF) for _ in range(2)]
    kp, vp = (t.clone().cuda() for t in pools)
    qo = torch.full((B, Hq, N, d), 7.0, dtype=BF, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = fa.kv_append(*split(c), kp, vp, table.cuda(), c["rule"], c["cu"]["off"], n_new.cuda(), qo, status)
    assert fa.check_status(status) == fa.OK and got is qo
    same = fa.qk_norm_rope(*split(c), c["rule"], q_offset=c["cu"]["off"])  # the same rows, pinned by its own tests
    want = [t.clone() for t in pools]
    for b in range(B):
        n = int(n_new[b])
        assert torch.equal(qo[b, :, :n], same[0][b, :, :n]) and (qo[b, :, n:] == 7).all()
        for i in range(n):
            p = int(c["off"][b]) + i
            for z in range(2):
                want[z][int(table[b, p // page]), :, p % page] = same[1 + z][b, :, i].cpu()
    assert torch.equal(kp.cpu(), want[0]) and torch.equal(vp.cpu(), want[1])
    # keys and values alone, as they are
    kp2, vp2 = (t.clone().cuda() for t in pools)
    _, k, v = split(c)
    assert fa.kv_append(None, k, v, kp2, vp2, table.cuda(), None, c["cu"]["off"], n_new.cuda(), status=status) is None
    assert torch.equal(vp2, vp) and (norm or rot or torch.equal(kp2, kp))


def expected_block(c, pools, scales, table, n_new, page):
    """What the 8-bit append leaves: (pages as e4m3 of the 64-bit rows, scales), and the rows themselves with their slack."""
    rows = expect(c)
    for z in range(2):
        y = rows[1 + z][0]
        for b in range(c["B"]):
            lo, n = int(c["off"][b]), int(n_new[b])
            for at in range(lo - lo % 32, lo + n, 32):
                i, j = max(at, lo), min(at + 32, lo + n)
                if j <= i:
                    continue
                pid, slot = int(table[b, at // page]), at % page
                x = y[b, i - lo:j - lo].transpose(0, 1)
                s = ref.need(x.abs().amax((1, 2)))
                was = scales[z][pid, :, slot // 32].double()
                now = torch.maximum(s, was) if i > at else s
                scales[z][pid, :, slot // 32] = now.float()
                old = pools[z][pid, :, slot:slot + i - at].float() * (was / now).float()[:, None, None]
                pools[z][pid, :, slot:slot + i - at] = old.to(F8)
                pools[z][pid, :, slot + i - at:slot + j - at] = (x / now[:, None, None]).clamp(-448, 448).float().to(F8)
    return rows


def fp8_pools(seed, total, Hkv, page, d):
    g = gen(seed)
    pools = [torch.randn(total, Hkv, page, d, generator=g).mul(40).to(F8) for _ in range(2)]
    scales = [torch.exp2(torch.randint(-9, -4, (total, Hkv, page // 32), generator=g).float()) for _ in range(2)]
    return pools, scales


@pytest.mark.parametrize("page,N,Hq,Hkv,d,rot,norm,offset", [
    (32, 1, 4, 2, 64, 64, True, 0), (128, 1, 32, 8, 128, 128, True, 31), (64, 1, 3, 3, 128, 48, False, 0),
    (64, 2, 4, 2, 128, 128, True, 30), (32, 100, 4, 1, 64, 32, True, 5), (128, 33, 8, 8, 128, 128, False, 0),
    (128, 200, 4, 2, 128, 0, True, 64)])
def test_append_fp8(page, N, Hq, Hkv, d, rot, norm, offset):
    B = 4
    c = make(13, B, N, Hq, Hkv, d, rot, norm, offset=offset)
    table, total = tables(14, B, -(-(offset + 50 + N) // page))
    n_new = torch.tensor([N, (N + 1) // 2, 0, N], dtype=torch.int32)
    pools, scales = fp8_pools(15, total, Hkv, page, d)
    kp, vp, ks, vs = (t.clone().cuda() for t in (*pools, *scales))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    qo = fa.kv_append_fp8(*split(c), kp, vp, ks, vs, table.cuda(), c["rule"], c["cu"]["off"], n_new.cuda(), status=status)
    assert fa.check_status(status) == fa.OK
    same = fa.qk_norm_rope(*split(c), c["rule"], q_offset=c["cu"]["off"])
    rows = expected_block(c, pools, scales, table, n_new, page)
    for b in range(B):
        assert torch.equal(qo[b, :, :int(n_new[b])], same[0][b, :, :int(n_new[b])])
    for z, (got, gs) in enumerate(((kp, ks), (vp, vs))):
        assert torch.equal(gs.cpu(), scales[z])
        got, want = got.cpu().float(), pools[z].float()
        # a new value is within half a step of the row's 64-bit value; all others are equal to the byte
        new = torch.zeros(got.shape, dtype=torch.bool)
        for b in range(B):
            for i in range(int(n_new[b])):
                p = int(c["off"][b]) + i
                pid, slot = int(table[b, p // page]), p % page
                new[pid, :, slot] = True
                s = scales[z][pid, :, slot // 32].double()[:, None]
                y, sl = rows[1 + z][0][b, i], rows[1 + z][1][b, i]
                err = (got[pid, :, slot].double() * s - y).abs()
                assert (err <= 2.0 ** -4 * y.abs() + 2.0 ** -10 * s + 2 * sl).all()
        assert torch.equal(got[~new], want[~new])


def test_append_fp8_token_by_token_then_cut_back():
    # a block filled one token at a time ends with the scale of its largest token; values that were rescaled on the way are
    # exact multiples of it (a power of two, no value near the subnormals' end), so they equal the block appended at once
    B, N, H, d, page = 1, 40, 2, 64, 64
    g = gen(16)
    x = torch.randn(B, N, 3 * H, d, generator=g)
    x *= torch.exp2(torch.arange(N) / 8).view(1, N, 1, 1)  # growing: several rescales
    x = x.sign() * x.abs().clamp(min=1.0)
    x = x.to(BF).cuda()
    q, k, v = x.split([H, H, H], dim=2)
    table = torch.tensor([[1]], dtype=torch.int32, device="cuda")
    pools = [[torch.zeros(2, H, page, d, device="cuda").to(F8) for _ in range(2)] + [torch.ones(2, H, 2, device="cuda") for _ in range(2)]
             for _ in range(2)]
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    fa.kv_append_fp8(q, k, v, *pools[0], table, q_offset=zero)
    for n in range(N):
        fa.kv_append_fp8(q[:, n:n + 1], k[:, n:n + 1], v[:, n:n + 1], *pools[1], table, q_offset=zero + n)
    for a, b in zip(pools[0][2:], pools[1][2:]):
        assert torch.equal(a, b)
    for (a, s), b in zip(((pools[0][0], pools[0][2]), (pools[0][1], pools[0][3])), pools[1][:2]):
        da, db = ref.dequant(a.cpu(), s.cpu()), ref.dequant(b.cpu(), s.cpu())
        # an early value was rounded under a smaller scale; under the last one it may be subnormal: half a step more
        assert ((da - db).abs() <= 2.0 ** -10 * s.cpu().double().repeat_interleave(32, -1)[..., None]).all()
    # cut back to 10 tokens and continue: the kept tokens do not move, the scale of the block does not shrink
    kept = pools[1][0][1, :, :10].clone()
    fa.kv_append_fp8(q[:, :3], k[:, :3], v[:, :3], *pools[1], table, q_offset=zero + 10)
    assert torch.equal(pools[1][0][1, :, :10].view(torch.uint8), kept.view(torch.uint8))
    assert torch.equal(pools[1][2], pools[0][2])


def test_append_fp8_extremes():
    # zeros, the smallest scale, infinities and NaN, and a block whose old scale is rubbish
    H, d, page = 1, 64, 32
    k = torch.zeros(4, 2, H, d)
    k[1] = 1e30
    k[2, 0, 0, 3], k[2, 0, 0, 4], k[2, 1] = float("inf"), float("nan"), 1.0
    k[3] = torch.randn(2, H, d, generator=gen(17))
    k = k.to(BF).cuda()
    table = torch.arange(4, dtype=torch.int32, device="cuda")[:, None].contiguous()
    for N, off in ((2, 0), (1, 3), (2, 3)):
        kp, vp = (torch.zeros(4, H, page, d, device="cuda").to(F8) for _ in range(2))
        ks, vs = (torch.full((4, H, 1), float("nan"), device="cuda") for _ in range(2))
        off_t = torch.full((4,), off, dtype=torch.int32, device="cuda")
        fa.kv_append_fp8(None, k[:, :N], k[:, :N], kp, vp, ks, vs, table, q_offset=off_t)
        assert ks[0, 0, 0] == 2.0 ** -40 and ks[1, 0, 0] == 2.0 ** 40 and ks[2, 0, 0] == 2.0 ** 40
        got = kp.float()
        assert not got[0].any() and (got[1, 0, off:off + N] == 448).all()
        assert got[2, 0, off, 3] == 448 and torch.isnan(got[2, 0, off, 4])
        y = k[3, :N, 0].double().cpu()
        s = float(ref.need(y.abs().max()))
        assert ks[3, 0, 0] == s
        assert ((got[3, 0, off:off + N].double().cpu() * s - y).abs() <= 2.0 ** -4 * y.abs() + 2.0 ** -10 * s).all()
        assert torch.equal(ks, vs)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("N", [1, 40])
def test_append_reports_bad_pages_positions_and_counts(fp8, N):
    H, d, page, B = 2, 64, 32, 5
    g = gen(18)
    k = torch.randn(B, N, H, d, generator=g).to(BF).cuda()
    table = torch.tensor([[0, 1, 2], [99, 99, 99], [-1, -1, -1], [3, 4, 5], [6, 7, 8]], dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 0, 0, 96, -32 * N], dtype=torch.int32, device="cuda")
    kp, vp = (torch.zeros(9, H, page, d, device="cuda").to(F8 if fp8 else BF) for _ in range(2))
    sc = [torch.ones(9, H, 1, device="cuda") for _ in range(2)] if fp8 else []
    call = fa.kv_append_fp8 if fp8 else fa.kv_append
    for only in range(B):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        n_new = torch.tensor([N if b == only else 0 for b in range(B)], dtype=torch.int32, device="cuda")
        call(None, k, k, kp, vp, *sc, table, q_offset=off, n_new=n_new, status=status)
        assert fa.check_status(status) == (fa.OK if only == 0 else fa.ERR_DEVICE_CHECK)
    assert not kp[3:].float().any() and kp[:2].float().any()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    n_new = torch.tensor([N + 1, -3, 0, 0, 0], dtype=torch.int32, device="cuda")
    call(None, k, k, kp, vp, *sc, table, q_offset=off, n_new=n_new, status=status)
    assert fa.check_status(status) == fa.ERR_DEVICE_CHECK


@pytest.mark.parametrize("N", [1, 2])
def test_append_fp8_many_requests_in_one_pool(N):
    # more requests than CTAs at a time, every one in a block of its own; the same values as one request at a time gives
    B, H, d, page = 3001, 1, 64, 32
    g = gen(22)
    x = torch.randn(B, N, 3 * H, d, generator=g).to(BF).cuda()
    q, k, v = x.split([H, H, H], dim=2)
    table = torch.randperm(B, generator=g).to(torch.int32)[:, None].contiguous().cuda()
    off = torch.randint(0, 31, (B,), generator=g).to(torch.int32).cuda()
    rule = fa.make_qk_rule(None, None, 0.0, inv_freq(64).cuda())
    kp, vp = (torch.zeros(B, H, page, d, device="cuda").to(F8) for _ in range(2))
    ks, vs = (torch.full((B, H, 1), 2.0 ** -40, device="cuda") for _ in range(2))
    fa.kv_append_fp8(q, k, v, kp, vp, ks, vs, table, rule, off)
    rows = fa.qk_norm_rope(None, k, None, rule, off)[1].transpose(1, 2).float()  # bf16 of the same rows
    pid = table[:, 0].long()
    b = torch.arange(B, device="cuda")
    for n in range(N):
        got_k = kp.float()[pid, 0, off.long() + n] * ks[pid, 0]
        got_v = vp.float()[pid, 0, off.long() + n] * vs[pid, 0]
        for got, want, s in ((got_k, rows[b, n, 0], ks[pid, 0]), (got_v, v[:, n, 0].float(), vs[pid, 0])):
            assert ((got - want).abs() <= (2.0 ** -4 + 2.0 ** -7) * want.abs() + 2.0 ** -9 * s).all()


def test_own_stream_and_captured_graph():
    c = make(19, 2, 1, 4, 2, 128, 128, True)
    page, d = 64, 128
    table = torch.arange(4, dtype=torch.int32).view(2, 2).cuda()
    x, off = c["cu"]["x"].clone(), torch.tensor([3, 70], dtype=torch.int32, device="cuda")
    pools = lambda: ([torch.zeros(4, 2, page, d, device="cuda").to(F8) for _ in range(2)] +
                     [torch.ones(4, 2, 2, device="cuda") for _ in range(2)])
    a, b = pools(), pools()
    qa = torch.zeros(2, 4, 1, d, dtype=BF, device="cuda")
    step = lambda p: fa.kv_append_fp8(*split(c, x), *p, table, c["rule"], off, q_out=qa)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(a)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step(a)
    torch.cuda.synchronize()
    for i in range(3):  # the captured step follows its inputs
        x.copy_(c["cu"]["x"] * (1 + i))
        off.copy_(torch.tensor([3 + i, 70 + i], dtype=torch.int32))
        graph.replay()
        q1 = qa.clone()
        step(b)
        torch.cuda.synchronize()
        assert torch.equal(q1, qa)
        for u, w in zip(a, b):
            assert np.array_equal(u.cpu().view(torch.uint8).numpy(), w.cpu().view(torch.uint8).numpy())


# ------------------------------------------------------------------------------------------ together with the attention
def test_training_run_through_the_attention():
    # projection rows -> attention -> loss <dO, O>, and back to the rows and the norm weights, against 64-bit autograd
    B, N, Hq, Hkv, d = 1, 200, 4, 2, 64
    c = make(20, B, N, Hq, Hkv, d, 64, True)
    q, k, v = fa.qk_norm_rope(*split(c), c["rule"], q_offset=c["cu"]["off"])
    bm = fa.create_block_mask(fa.make_mask_rule([("causal",)]), B, Hq, N, N, 128, 128)
    out, lse = fa.flex_forward(q, k, v, bm, out_dtype=F32)
    dout = torch.randn(B, Hq, N, d, generator=gen(21)).to(BF)
    dq, dk, dv = fa.flex_backward(q, k, v, out, lse, dout.cuda(), bm)
    a, b, _ = split(c)
    got = fa.qk_norm_rope_backward(a, b, dq, dk, dv, c["rule"], q_offset=c["cu"]["off"], grad_dtype=F32)
    x = c["x"].double().requires_grad_()
    wq, wk = c["wq"].double().requires_grad_(), c["wk"].double().requires_grad_()
    xs = x.split([Hq, Hkv, Hkv], dim=2)
    rows = [ref.rotate(xx * torch.rsqrt(xx.square().mean(-1, keepdim=True) + c["eps"]) * w, c["pos"], c["f"], False).transpose(1, 2)
            for xx, w in zip(xs, (wq, wk))]
    kk, vv = (t.repeat_interleave(Hq // Hkv, 1) for t in (rows[1], xs[2].transpose(1, 2)))
    s = (rows[0] @ kk.transpose(-1, -2) / d ** 0.5).masked_fill(torch.ones(N, N).triu(1).bool(), -torch.inf)
    (torch.softmax(s, -1) @ vv).mul(dout.double()).sum().backward()
    # the attention's own bound (2e-2 of the largest value, its bf16 products) times the norm of the weighted rotation
    # (at most the weight times r sqrt(2), within the largest value's scale), plus q and k rounded once to bf16
    for g, w in zip((torch.cat(got[:3], 2), got[3], got[4]), (x.grad, wq.grad, wk.grad)):
        assert (g.double().cpu() - w).abs().max() <= 4e-2 * w.abs().max()


def test_rows_past_32_bit_offsets():
    # a projection of more than 2^31 elements: its last tokens come out as those of a short one at the same positions
    N, n, Hq, Hkv, d = 350001, 5, 32, 8, 128
    c = make(60, 1, n, Hq, Hkv, d, 128, True)
    x = torch.zeros(1, N, Hq + 2 * Hkv, d, dtype=BF, device="cuda")
    assert x.numel() > 2 ** 31
    x[:, N - n:] = c["cu"]["x"]
    shift = torch.tensor([N - n], dtype=torch.int32, device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    long = fa.qk_norm_rope(*split(c, x), c["rule"], q_offset=zero)
    short = fa.qk_norm_rope(*split(c), c["rule"], q_offset=shift)
    for a, b in zip(long, short):
        assert torch.equal(a[:, :, N - n:], b) and not a[:, :, :8].any()
    g = gen(61)
    dy = [torch.randn(1, h, n, d, generator=g).cuda() for h in (Hq, Hkv, Hkv)]
    far = [torch.zeros(1, h, N, d, device="cuda") for h in (Hq, Hkv, Hkv)]
    for a, b in zip(far, dy):
        a[:, :, N - n:] = b
    q, k, _ = split(c, x)
    grad = torch.empty_like(x)
    got = fa.qk_norm_rope_backward(q, k, *far, c["rule"], q_offset=zero, **dict(zip(("dq_in", "dk_in", "dv_in"), split(c, grad))))
    q, k, _ = split(c)
    want = fa.qk_norm_rope_backward(q, k, *dy, c["rule"], q_offset=shift)
    for a, b in zip(got[:3], want[:3]):
        assert torch.equal(a[:, N - n:], b) and not a[:, :8].any()
    for a, b in zip(got[3:], want[3:]):  # other CTAs hold the rows: the same terms in another order
        assert ((a - b).abs() <= 1e-5 * b.abs().max()).all()
