"""Norms of queries and keys with the rotary positions: orthros_norm_rotate, its gradient and
orthros_norm_rotate_append against plain fp64 formulas.

Tolerances, in units of e = 2^-24. The sum of d squares runs in at most 16 + 5 additions a lane, so it
is off by 22 e, its root by half of that, rsqrtf by 2 ulp (4 e), so r = 1/rms by 16 e; xh = x r by 17, a = alpha w
by 1, the affine's fma by 1: u by 20 e (|a xh| + |beta|), and the rotation adds 12 e (|u_a| + |u_b|)
(test_rotary.py), so y is off by 32 e times the rotated magnitudes, plus half a step of its type.
Backward: g by 12 e |g|*, |g|* the rotated magnitudes of dy; u = a g by 14 e, mean(u xh) by the 14 + 17
of its terms, 22 of its sum and 2 of its factors, 55 e mean(|a g* xh|); dx = r (u - xh mean) by at
most 96 e r (|a| g* + |xh| mean(|a| g* |xh|)) with xh's 17, r's 16 and the fma's, plus half a step.
Sums over n tokens (and H heads): their terms' 12 + 17 + 2 and at most n + H additions, the factor's 1.
"""
import numpy as np
import pytest
import torch

import efficient_long_context_gb300 as ola
from tests.test_rotary import HALF_STEP, frequencies, make, plain_rotate

E = 2.0 ** -24
EPS = 1e-5
P = 1 << 12  # a 16-byte aligned address that no refused call reads


@pytest.fixture(scope="module")
def lib():
    from efficient_long_context_gb300 import build

    build.build()
    return ola.load_library()


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------
def _rotate(lib, **o):
    a = dict(x=P, xs=256, pos=P, w=P, eps=EPS, al=None, be=None, st=P, rot=64, lay=0, amp=1.0, n=2, H=4, d=64, dt=0, y=2 * P,
             ys=256)
    a.update(o)
    return lib.orthros_norm_rotate(a["x"], a["xs"], a["pos"], a["w"], a["eps"], a["al"], a["be"], a["st"], a["rot"], a["lay"],
                                   a["amp"], a["n"], a["H"], a["d"], a["dt"], a["y"], a["ys"], None)


@pytest.mark.parametrize("over,code", [
    (dict(eps=0.0), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(w=P + 4), 1),
    (dict(n=-1), 1), (dict(H=0), 1), (dict(dt=7), 1), (dict(d=96), 2), (dict(rot=66), 1), (dict(rot=40), 2), (dict(lay=2), 1),
    (dict(st=None), 1), (dict(al=P), 1), (dict(x=None), 1), (dict(x=P + 8), 1), (dict(xs=260), 1), (dict(ys=248), 1),
    (dict(y=P, xs=512), 1), (dict(pos=None), 1)])
def test_rotate_refusals(lib, over, code):
    assert _rotate(lib, **over) == code
    assert ola.orthros_last_error() != ""


def _backward(lib, **o):
    a = dict(dy=P, dys=256, x=P, xs=256, pos=P, w=P, eps=EPS, al=P, st=P, rot=64, lay=0, amp=1.0, n=2, H=4, d=64, dt=0,
             dx=2 * P, dxs=256, dw=P, da=P, db=P, ws=P, wsb=1 << 24)
    a.update(o)
    return lib.orthros_norm_rotate_backward(
        a["dy"], a["dys"], a["x"], a["xs"], a["pos"], a["w"], a["eps"], a["al"], a["st"], a["rot"], a["lay"], a["amp"], a["n"],
        a["H"], a["d"], a["dt"], a["dx"], a["dxs"], a["dw"], a["da"], a["db"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("over,code", [
    (dict(eps=0.0), 1), (dict(w=P + 8), 1), (dict(n=-1), 1), (dict(d=32), 2), (dict(al=P + 4), 1), (dict(da=None), 1),
    (dict(ws=None), 4), (dict(da=None, db=None, ws=None), 4), (dict(wsb=64), 4), (dict(ws=P + 16), 1), (dict(dy=None), 1),
    (dict(x=None), 1), (dict(x=None, dw=None, da=None, db=None), 1), (dict(dxs=128), 1), (dict(dx=P, dxs=512), 1),
    (dict(pos=None), 1)])
def test_backward_refusals(lib, over, code):
    assert _backward(lib, **over) == code


def _append(lib, **o):
    a = dict(q=P, qs=256, qo=P, qos=256, k=P, ks=128, v=P, vs=128, qw=P, kw=P, eps=EPS, ab=None, bb=None, ao=None, bo=None,
             st=P, rot=64, lay=0, amp=1.0, sl=P, tp=P, op=P, nn=2, no=1, Hq=4, Hkv=2, d=64, dt=0, qr=P, qor=P, kc=P, vc=P,
             ps=16, np_=4, ws=P, wsb=256)
    a.update(o)
    return lib.orthros_norm_rotate_append(
        a["q"], a["qs"], a["qo"], a["qos"], a["k"], a["ks"], a["v"], a["vs"], a["qw"], a["kw"], a["eps"], a["ab"], a["bb"],
        a["ao"], a["bo"], a["st"], a["rot"], a["lay"], a["amp"], a["sl"], a["tp"], a["op"], a["nn"], a["no"], a["Hq"], a["Hkv"],
        a["d"], a["dt"], a["qr"], a["qor"], a["kc"], a["vc"], a["ps"], a["np_"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("over,code", [
    (dict(eps=0.0), 1), (dict(eps=0.0, qw=None), 1), (dict(eps=-1.0), 1), (dict(qw=P + 4), 1), (dict(kw=P + 4), 1),
    (dict(nn=-1), 1), (dict(no=-1), 1), (dict(Hkv=0), 1), (dict(d=80), 2), (dict(dt=3), 1), (dict(st=None), 1), (dict(ab=P), 1),
    (dict(ws=None), 4), (dict(ws=P + 64), 1), (dict(k=None), 1), (dict(v=P + 4), 1), (dict(qr=None), 1), (dict(sl=None), 1),
    (dict(tp=None), 1), (dict(kc=None), 1), (dict(vc=P + 8), 1), (dict(ps=0), 1), (dict(np_=0), 1), (dict(qo=None), 1),
    (dict(qor=None), 1), (dict(op=None), 1)])
def test_append_refusals(lib, over, code):
    assert _append(lib, **over) == code


def test_binding_refusals(lib):
    x, pos, st = torch.zeros(3, 4, 64), torch.zeros(3, dtype=torch.int32), torch.zeros(32, dtype=torch.int64)
    for bad in (dict(weight=torch.zeros(4, 64)), dict(weight=torch.zeros(64, dtype=torch.bfloat16)), dict(layout="x"),
                dict(out=torch.zeros(2, 4, 64)), dict(alpha=torch.zeros(64))):
        with pytest.raises(ola.OrthrosError):
            ola.orthros_norm_rotate(x, pos, st, **bad)
    with pytest.raises(ola.OrthrosError):
        ola.orthros_norm_rotate(x, pos, st)  # not on the GPU
    k = torch.zeros(2, 16, 4, 64)
    for eps in (1e-50, -1.0, float("nan")):  # 0 in 32 bits is not "no norm"
        with pytest.raises(ola.OrthrosError):
            ola.orthros_norm_rotate_append(None, x, x, k, k, pos, pos, st, eps=eps)


def test_workspace_size(lib):
    f = ola.orthros_norm_rotate_backward_workspace_size
    assert f(100, 4, 64) > ola.orthros_rotate_backward_workspace_size(100, 4, 64) > 0
    assert f(0, 4, 64) > 0 and f(-1, 4, 64) == 0 and f(4, 4, 96) == 0 and f(4, 0, 64) == 0


# ---------------------------------------------------------------------------
# plain forms, fp64 on the CPU
# ---------------------------------------------------------------------------
def plain_norm(x, w, al, be):
    """(u, |a xh| + |beta|, r, xh) of the affine of a normed x [n, H, d]."""
    x = x.double()
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    xh = x * r
    z = xh if w is None else xh * w.double()
    if al is None:
        return z, z.abs(), r, xh
    return z * al.double() + be.double(), (z * al.double()).abs() + be.double().abs(), r, xh


def close(got, ref, tol, what):
    g = got.double().cpu()
    assert g.shape == ref.shape and bool(torch.isfinite(g).all()), what
    d = (g - ref).abs() / (tol + 1e-37)
    assert float(d.max() if d.numel() else 0) <= 1, f"{what}: {float(d.max()):.3f} of the tolerance"


def check_rows(got, x, w, al, be, pos, steps, layout, amp, what):
    u, mag_u, _, _ = plain_norm(x, w, al, be)
    ref, _ = plain_rotate(u, pos, steps, layout, amp)
    _, mag = plain_rotate(mag_u, pos, steps, layout, amp)
    close(got, ref, HALF_STEP[got.dtype] * ref.abs() + 32 * E * mag, what)


def weight(d, seed):
    return 1.0 + 0.3 * torch.randn(d, generator=torch.Generator().manual_seed(seed))


SHAPES = [(1, 1, 64, 64), (1, 32, 128, 128), (17, 3, 64, 16), (33, 5, 128, 48), (130, 32, 128, 128), (515, 12, 128, 96),
          (64, 40, 64, 32), (7, 33, 128, 64)]


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n,H,d,rot", SHAPES)
def test_norm_rotate(n, H, d, rot, dtype, layout):
    x, al, be, pos = make(n, H, d, dtype, seed=n + H)
    x[n // 2] *= 100.0
    steps = ola.orthros_rotary_steps(frequencies(rot))
    amp = 1.25
    for w in (None, weight(d, n)):
        for aff in ((None, None), (al, be)):
            kw = dict(alpha=al.cuda(), beta=be.cuda()) if aff[0] is not None else {}
            y = ola.orthros_norm_rotate(x.cuda(), pos.cuda(), steps.cuda(), None if w is None else w.cuda(), EPS, layout=layout,
                                        amplitude=amp, **kw)
            check_rows(y, x, w, *aff, pos, steps, layout, amp, f"w={w is not None} affine={bool(kw)}")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_strides_in_place_and_zero_rows(dtype):
    n, Hq, Hkv, d = 37, 6, 2, 64
    g = torch.Generator().manual_seed(3)
    packed = torch.randn(n, Hq + 2 * Hkv, d, generator=g).to(dtype).cuda()
    pos = torch.randint(0, 5000, (n,), generator=g, dtype=torch.int32).cuda()
    steps, w = ola.orthros_rotary_steps(frequencies(32)).cuda(), weight(d, 1).cuda()
    before = packed.clone()
    want_q = ola.orthros_norm_rotate(packed[:, :Hq].contiguous(), pos, steps, w)
    want_k = ola.orthros_norm_rotate(packed[:, Hq:Hq + Hkv].contiguous(), pos, steps, w)
    assert torch.equal(ola.orthros_norm_rotate(packed[:, :Hq], pos, steps, w), want_q)
    k = packed[:, Hq:Hq + Hkv]
    ola.orthros_norm_rotate(k, pos, steps, w, out=k)
    assert torch.equal(k, want_k) and torch.equal(packed[:, :Hq], before[:, :Hq])
    assert torch.equal(packed[:, Hq + Hkv:], before[:, Hq + Hkv:])
    assert ola.orthros_norm_rotate(packed[:0, :Hq], pos[:0], steps, w).shape == (0, Hq, d)
    # a row of zeros has no direction: its norm is zero, and so is its output
    z = torch.zeros(2, 3, d, dtype=dtype, device="cuda")
    assert torch.equal(ola.orthros_norm_rotate(z, pos[:2], steps, w), z)
    dx, dw, _, _ = ola.orthros_norm_rotate_backward(z, z, pos[:2], steps, w, affine_grads=False)
    assert torch.equal(dx, z) and not bool(dw.any())


@pytest.mark.gpu
def test_non_finite_rows_stay_in_their_rows():
    n, H, d = 20, 6, 128
    x, al, be, pos = make(n, H, d, torch.bfloat16, seed=4)
    steps = ola.orthros_rotary_steps(frequencies(64)).cuda()
    kw = dict(alpha=al.cuda(), beta=be.cuda())
    want = ola.orthros_norm_rotate(x.cuda(), pos.cuda(), steps, **kw)
    x[3, 2, 5], x[7, 0, 0] = float("nan"), float("inf")
    got = ola.orthros_norm_rotate(x.cuda(), pos.cuda(), steps, **kw)
    keep = torch.ones(n, H, dtype=torch.bool)
    keep[3, 2] = keep[7, 0] = False
    assert torch.equal(got[keep.cuda()], want[keep.cuda()])
    assert bool(torch.isnan(got[3, 2]).all()) and bool(torch.isnan(got[7, 0, 0]))


# ---------------------------------------------------------------------------
# gradients
# ---------------------------------------------------------------------------
def check_backward(got, dy, x, w, al, pos, steps, layout, amp, what):
    n, H, d = x.shape
    dx, dw, da, db = got
    g, mag = plain_rotate(dy.double(), pos, steps, layout, amp, sign=-1.0)
    _, _, r, xh = plain_norm(x, None, None, None)
    one = torch.ones(d, dtype=torch.float64)
    ww = one if w is None else w.double()
    a = ww.expand(H, d) if al is None else al.double() * ww
    u = a * g
    ref = r * (u - xh * (u * xh).mean(-1, keepdim=True))
    m = a.abs() * mag
    close(dx, ref, HALF_STEP[dx.dtype] * ref.abs() + 96 * E * r * (m + xh.abs() * (m * xh.abs()).mean(-1, keepdim=True)), what + " dx")
    S, T = (g * xh).sum(0), (mag * xh.abs()).sum(0)
    k = (n + H + 64) * E
    if dw is not None:
        at = torch.ones(H, d, dtype=torch.float64) if al is None else al.double()
        close(dw, (at * S).sum(0), k * (at.abs() * T).sum(0), what + " dw")
    if da is not None:
        close(da, S * ww, k * T * ww.abs(), what + " d_alpha")
        close(db, g.sum(0), k * mag.sum(0), what + " d_beta")


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n,H,d,rot", SHAPES + [(2100, 4, 64, 64), (300, 130, 128, 128)])
def test_backward(n, H, d, rot, dtype, layout):
    x, al, _, pos = make(n, H, d, dtype, seed=7 * n + H)
    dy = torch.randn(n, H, d, generator=torch.Generator().manual_seed(n)).to(dtype)
    w = weight(d, H)
    w[1] = 0.0  # a channel that is switched off still has a gradient of its weight
    steps = ola.orthros_rotary_steps(frequencies(rot))
    amp = 0.75
    args = (dy.cuda(), x.cuda(), pos.cuda(), steps.cuda())
    kw = dict(layout=layout, amplitude=amp)
    ref = (dy, x, w, al, pos, steps, layout, amp)
    got = ola.orthros_norm_rotate_backward(*args, w.cuda(), EPS, alpha=al.cuda(), **kw)
    check_backward(got, *ref, "all")
    again = ola.orthros_norm_rotate_backward(*args, w.cuda(), EPS, alpha=al.cuda(), **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    # parts of the gradients are the same bits
    some = ola.orthros_norm_rotate_backward(*args, w.cuda(), EPS, alpha=al.cuda(), affine_grads=False, **kw)
    assert torch.equal(some[0], got[0]) and torch.equal(some[1], got[1]) and some[2] is None
    some = ola.orthros_norm_rotate_backward(*args, w.cuda(), EPS, alpha=al.cuda(), weight_grad=False, **kw)
    assert torch.equal(some[0], got[0]) and some[1] is None and torch.equal(some[2], got[2]) and torch.equal(some[3], got[3])
    some = ola.orthros_norm_rotate_backward(*args, w.cuda(), EPS, alpha=al.cuda(), weight_grad=False, affine_grads=False, **kw)
    assert torch.equal(some[0], got[0]) and some[1] is None and some[2] is None
    # neither weight nor affine in the forward; in place over dy
    check_backward(ola.orthros_norm_rotate_backward(*args, None, EPS, **kw), dy, x, None, None, pos, steps, layout, amp, "bare")
    own = args[0].clone()
    dx, _, _, _ = ola.orthros_norm_rotate_backward(own, *args[1:], w.cuda(), EPS, alpha=al.cuda(), out=(own, None, None, None), **kw)
    assert dx.data_ptr() == own.data_ptr() and torch.equal(own, got[0])


@pytest.mark.gpu
def test_backward_of_no_tokens():
    x = torch.zeros(0, 4, 64, device="cuda")
    pos, steps = torch.zeros(0, dtype=torch.int32, device="cuda"), ola.orthros_rotary_steps(frequencies(64)).cuda()
    out = [x, torch.ones(64, device="cuda"), torch.ones(4, 64, device="cuda"), torch.ones(4, 64, device="cuda")]
    ola.orthros_norm_rotate_backward(x, x, pos, steps, out=out)
    assert not any(bool(t.any()) for t in out[1:])


@pytest.mark.gpu
def test_backward_against_differences():
    """Central differences in fp64 of sum(w . y) of the definition along random directions; the step's own
    error is a third of what doubling the step changes."""
    n, H, d, rot = 29, 3, 64, 48
    x, al, be, pos = make(n, H, d, torch.float32, seed=5)
    g = torch.Generator().manual_seed(6)
    wt, dy = weight(d, 2), torch.randn(n, H, d, generator=g)
    steps = ola.orthros_rotary_steps(frequencies(rot))
    got = ola.orthros_norm_rotate_backward(dy.cuda(), x.cuda(), pos.cuda(), steps.cuda(), wt.cuda(), EPS, alpha=al.cuda())

    def loss(v):
        u, _, _, _ = plain_norm(v["x"], v["w"], v["al"], v["be"])
        return float((dy.double() * plain_rotate(u, pos, steps, "half", 1.0)[0]).sum())

    base = dict(x=x.double(), w=wt.double(), al=al.double(), be=be.double())
    for name, grad in zip(("x", "w", "al", "be"), got):
        e = torch.randn(base[name].shape, generator=g, dtype=torch.float64)

        def diff(h):
            return (loss(dict(base, **{name: base[name] + h * e})) - loss(dict(base, **{name: base[name] - h * e}))) / (2 * h)

        num, ana = diff(1e-4), float((grad.double().cpu() * e).sum())
        # fp32 gradients: each term 128 e of magnitudes no larger than 8 |dy| (w, alpha, xh of normal size)
        noise = 128 * E * 8 * float(dy.abs().sum()) + abs(diff(2e-4) - num) + 1e-7
        assert abs(num - ana) <= noise, (name, num, ana, noise)


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n,n_out,Hq,Hkv,d,page,rot", [(1, 1, 1, 1, 64, 1, 16), (32, 32, 32, 8, 128, 64, 128), (70, 3, 12, 4, 64, 5, 48),
                                                       (300, 0, 8, 2, 128, 16, 64), (0, 4, 4, 4, 64, 8, 64)])
def test_append(n, n_out, Hq, Hkv, d, page, rot, dtype, layout):
    g = torch.Generator().manual_seed(n + Hq)
    packed = torch.randn(n, Hq + 2 * Hkv, d, generator=g).to(dtype)
    q, k, v = packed[:, :Hq], packed[:, Hq:Hq + Hkv], packed[:, Hq + Hkv:]
    qo = torch.randn(n_out, Hq, d, generator=g).to(dtype)
    pos, opos = (torch.randint(0, 100000, (m,), generator=g, dtype=torch.int32) for m in (n, n_out))
    pages = (n + page - 1) // page + 3
    slots = torch.randperm(pages * page, generator=g)[:n].to(torch.int32)
    if n > 4:
        slots[::5] = -1  # rows of padding
    kc, vc = (torch.randn(pages, page, Hkv, d, generator=g).to(dtype) for _ in range(2))
    qw, kw = weight(d, 1), weight(d, 2)
    aff = [1 + 0.1 * torch.randn(Hq, d, generator=g), 0.1 * torch.randn(Hq, d, generator=g)]
    affo = [1 + 0.1 * torch.randn(Hq, d, generator=g), 0.1 * torch.randn(Hq, d, generator=g)]
    steps = ola.orthros_rotary_steps(frequencies(rot))
    amp = 1.1
    dev = packed.cuda()
    parts = (dev[:, :Hq], dev[:, Hq:Hq + Hkv], dev[:, Hq + Hkv:])
    ws = torch.full((256,), 255, dtype=torch.uint8, device="cuda")
    for norm in (True, False):
        kcd, vcd = kc.cuda(), vc.cuda()
        extra = dict(eps=EPS, q_weight=qw.cuda(), k_weight=kw.cuda()) if norm else dict(eps=0.0)
        qr, qor = ola.orthros_norm_rotate_append(
            *parts, kcd, vcd, slots.cuda(), pos.cuda(), steps.cuda(), layout=layout, amplitude=amp,
            q_out=qo.cuda() if n_out else None, out_positions=opos.cuda() if n_out else None, alpha_base=aff[0].cuda(),
            beta_base=aff[1].cuda(), alpha_out=affo[0].cuda(), beta_out=affo[1].cuda(), workspace=ws, **extra)
        assert ola.orthros_check(ws) == (0, 0)
        at = slots >= 0
        rows = slots[at].long()
        want_v = vc.flatten(0, 1).clone()
        want_v[rows] = v[at]
        assert torch.equal(vcd.cpu().flatten(0, 1), want_v)
        rest = torch.ones(pages * page, dtype=torch.bool)
        rest[rows] = False
        kg = kcd.cpu().flatten(0, 1)
        assert torch.equal(kg[rest], kc.flatten(0, 1)[rest])
        if norm:
            check_rows(qr, q, qw, *aff, pos, steps, layout, amp, "q")
            check_rows(kg[rows], k[at], kw, None, None, pos[at], steps, layout, amp, "k")
            if n_out:
                check_rows(qor, qo, qw, *affo, opos, steps, layout, amp, "q_out")
        else:  # the bits of the calls without a norm
            rope = dict(layout=layout, amplitude=amp)
            assert torch.equal(qr, ola.orthros_rotate(parts[0], pos.cuda(), steps.cuda(), alpha=aff[0].cuda(), beta=aff[1].cuda(), **rope))
            assert torch.equal(kg[rows], ola.orthros_rotate(parts[1], pos.cuda(), steps.cuda(), **rope).cpu()[at])


@pytest.mark.gpu
def test_append_flags_bad_slots():
    n, Hkv, d, page, pages = 6, 2, 64, 8, 2
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(n, Hkv, d, generator=g).cuda() for _ in range(2))
    pos, steps = torch.arange(n, dtype=torch.int32).cuda(), ola.orthros_rotary_steps(frequencies(64)).cuda()
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    for bad, bits in ((-1, 0), (pages * page, 2), (-2, 2), (2 ** 31 - 1, 2), (-2 ** 31, 2), (pages * page - 1, 0)):
        kc = torch.zeros(pages + 1, page, Hkv, d, device="cuda")  # the last page is behind the pool
        vc = torch.zeros_like(kc)
        slots = torch.tensor([0, 5, bad, 9, 1, 7], dtype=torch.int32).cuda()
        ola.orthros_norm_rotate_append(None, k, v, kc[:pages], vc[:pages], slots, pos, steps, workspace=ws)
        assert ola.orthros_check(ws) == (5 if bits else 0, bits)
        rows = [0, 5, 9, 1, 7]
        want = torch.zeros((pages + 1) * page, Hkv, d, device="cuda")
        want[rows] = v[[0, 1, 3, 4, 5]]
        if bad == pages * page - 1:
            want[bad] = v[2]
        assert torch.equal(vc.flatten(0, 1), want)


@pytest.mark.gpu
def test_graph_replay_and_stream_argument():
    """The calls captured once follow their inputs; a stream= call runs on that stream."""
    n, H, d = 40, 8, 128
    x, al, be, pos = make(n, H, d, torch.bfloat16, seed=9)
    xd, posd, steps, w = x.cuda(), pos.cuda(), ola.orthros_rotary_steps(frequencies(128)).cuda(), weight(d, 3).cuda()
    ald, bed = al.cuda(), be.cuda()
    ws = torch.empty(ola.orthros_norm_rotate_backward_workspace_size(n, H, d), dtype=torch.uint8, device="cuda")

    def both(**kw):
        y = ola.orthros_norm_rotate(xd, posd, steps, w, alpha=ald, beta=bed, **kw)
        return (y, *ola.orthros_norm_rotate_backward(y, xd, posd, steps, w, alpha=ald, workspace=ws, **kw))

    want = both()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for scale in (1.0, 3.0):
        xd.copy_(x.cuda() * scale)
        want = [t.clone() for t in both()]
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = both(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d,rot", [(64, 32), (128, 128)])
def test_rows_whose_squares_overflow_have_no_direction(d, rot, dtype, layout):
    """A head whose sum of squares is past fp32's range has xh = 0: the forward gives its rotated beta, the
    gradient of x is 0 there, whatever the products of x and dy come to, and no sum takes anything of it."""
    n, H = 9, 3
    x, al, be, pos = make(n, H, d, dtype, seed=21)
    dy = torch.randn(n, H, d, generator=torch.Generator().manual_seed(22)).to(dtype)
    big = [(2, 1, 1.5e38), (5, 0, 3e30), (7, 2, -2e38)]
    for i, h, v in big:
        x[i, h] = v
        dy[i, h] = 64.0  # v dy is past 3.4e38 for two of them
    x[7, 2, ::2] = 2e38  # products of both signs
    steps, w = ola.orthros_rotary_steps(frequencies(rot)), weight(d, 4)
    kw = dict(layout=layout, alpha=al.cuda())
    y = ola.orthros_norm_rotate(x.cuda(), pos.cuda(), steps.cuda(), w.cuda(), EPS, beta=be.cuda(), **kw)
    got = ola.orthros_norm_rotate_backward(dy.cuda(), x.cuda(), pos.cuda(), steps.cuda(), w.cuda(), EPS, **kw)
    zero = x.clone()
    for i, h, _ in big:
        zero[i, h] = 0  # rows whose norm is 0 as well
        assert not bool(got[0][i, h].any())
    want = ola.orthros_norm_rotate_backward(dy.cuda(), zero.cuda(), pos.cuda(), steps.cuda(), w.cuda(), EPS, **kw)
    rows = torch.ones(n, H, dtype=torch.bool)
    for i, h, _ in big:
        rows[i, h] = False
    assert torch.equal(got[0][rows.cuda()], want[0][rows.cuda()])
    assert all(torch.equal(a, b) for a, b in zip(got[1:], want[1:]))
    assert torch.equal(y, ola.orthros_norm_rotate(zero.cuda(), pos.cuda(), steps.cuda(), w.cuda(), EPS, beta=be.cuda(), **kw))
