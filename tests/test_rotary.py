"""Rotary positions: orthros_rotary_frequencies, orthros_rotary_steps (host),
orthros_rotate, orthros_rotate_backward and orthros_rotate_append against plain
fp64 formulas.

Tolerances. Angles: the phase is exact to 2^-32 turn, its float form is off by
half an ulp of at most pi (pi 2^-24), sincospif by 2 ulp of at most 1, so cos
and sin are off by less than 6 * 2^-24. Each output is two products and a sum
(3 roundings, 2^-24 each) of values that went through the affine (2 more):
|err| <= 12 * 2^-24 * amplitude * (|u_a| + |u_b|), u bounded by |alpha x| + |beta|,
plus half a step of the element type (2^-8 |y| for bf16, 2^-24 |y| for fp32).
Sums over n tokens add at most (depth + 12) 2^-24 sum |terms|, depth <= n.
"""
import ctypes
import math

import numpy as np
import pytest
import torch

import efficient_long_context_gb300 as ola

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
ANGLE = 12 * 2.0 ** -24


@pytest.fixture(scope="module")
def lib():
    from efficient_long_context_gb300 import build

    build.build()
    return ola.load_library()


# ---------------------------------------------------------------------------
# plain forms, fp64 on the CPU
# ---------------------------------------------------------------------------
def exact_angles(pos, steps):
    """cos, sin [n, pairs] in fp64 of the phases the steps define (integer products modulo a turn)."""
    st = [int(s) % 2 ** 64 for s in steps.tolist()]
    ph = np.array([[((int(t) * s) % 2 ** 64) / 2.0 ** 64 for s in st] for t in pos.tolist()]).reshape(len(pos), len(st))
    return torch.from_numpy(np.cos(2 * np.pi * ph)), torch.from_numpy(np.sin(2 * np.pi * ph))


def channels(rot, layout):
    return (list(range(rot // 2)), list(range(rot // 2, rot))) if layout == "half" else \
        (list(range(0, rot, 2)), list(range(1, rot, 2)))


def plain_rotate(u, pos, steps, layout, amp, sign=1.0):
    """u [n, H, d] fp64 -> (rotated, |u_a| + |u_b| per channel)."""
    c, s = exact_angles(pos, steps)
    c, s = amp * c[:, None, :], amp * sign * s[:, None, :]
    ia, ib = channels(2 * steps.numel(), layout)
    y, mag = u.clone(), u.abs()
    y[..., ia] = u[..., ia] * c - u[..., ib] * s
    y[..., ib] = u[..., ia] * s + u[..., ib] * c
    m = amp * (mag[..., ia] + mag[..., ib])
    mag[..., ia], mag[..., ib] = m, m
    return y, mag


def check(got, ref, mag, dtype, what, extra=0.0):
    g = got.double().cpu()
    tol = HALF_STEP[dtype] * ref.abs() + ANGLE * mag + extra + 1e-37
    bad = (g - ref).abs() > tol
    assert g.shape == ref.shape and not bool(bad.any()) and bool(torch.isfinite(g).all()), \
        f"{what}: worst {((g - ref).abs() / tol).max():.3f} of the tolerance, {int(bad.sum())} elements"


def frequencies(rot):
    f, _ = ola.orthros_rotary_frequencies(rot, 10000.0)
    return f


# ---------------------------------------------------------------------------
# host: frequencies, steps, refusals
# ---------------------------------------------------------------------------
def test_frequency_rules(lib):
    rot, base, fac, L = 64, 10000.0, 8.0, 8192.0
    i = np.arange(rot // 2)
    f = base ** (-2.0 * i / rot)
    got, amp = ola.orthros_rotary_frequencies(rot, base)
    np.testing.assert_allclose(got, f, rtol=1e-15)
    assert amp == 1.0
    np.testing.assert_allclose(ola.orthros_rotary_frequencies(rot, base, "linear", factor=fac)[0], f / fac, rtol=1e-15)
    st = ola.orthros_rotary_frequencies(rot, base, "stretch", factor=fac)[0].numpy()
    np.testing.assert_allclose(st[0], f[0], rtol=1e-15)           # the highest frequency stays
    np.testing.assert_allclose(st[-1], f[-1] / fac, rtol=1e-12)   # the lowest is divided by the factor
    b, amp = ola.orthros_rotary_frequencies(rot, base, "bands", factor=fac, original_length=L, low_turns=1, high_turns=4)
    turns = L * f / (2 * math.pi)
    b = b.numpy()
    np.testing.assert_allclose(b[turns >= 4], f[turns >= 4], rtol=1e-15)
    np.testing.assert_allclose(b[turns <= 1], f[turns <= 1] / fac, rtol=1e-15)
    mid = (turns > 1) & (turns < 4)
    assert mid.any() and np.all(b[mid] < f[mid]) and np.all(b[mid] > f[mid] / fac) and np.all(np.diff(b) < 0)
    t, amp = ola.orthros_rotary_frequencies(rot, base, "bands_tempered", factor=fac, original_length=L)
    np.testing.assert_allclose(t, b, rtol=1e-15)
    assert amp == np.float32(0.1 * math.log(fac) + 1.0)


@pytest.mark.parametrize("kw", [dict(rot_dim=3), dict(rot_dim=0), dict(base=1.0), dict(base=float("nan")),
                                dict(scaling="linear", factor=0.5), dict(scaling="linear", factor=float("inf")),
                                dict(rot_dim=2, scaling="stretch", factor=2.0),
                                dict(scaling="bands", factor=8.0, original_length=0.0),
                                dict(scaling="bands", factor=8.0, original_length=10.0, low_turns=4, high_turns=4),
                                dict(scaling="unknown")])
def test_frequency_refusals(lib, kw):
    a = dict(rot_dim=64, base=10000.0, scaling="plain")
    a.update(kw)
    with pytest.raises(ola.OrthrosError):
        ola.orthros_rotary_frequencies(a.pop("rot_dim"), a.pop("base"), a.pop("scaling"), **a)


def test_steps_are_the_turns(lib):
    f = [1.0, 0.5, 1e-3, 0.0, 2 * math.pi, -1.0, 2 * math.pi + 1.0, 1e-12, -1e-30]
    st = [int(s) % 2 ** 64 for s in ola.orthros_rotary_steps(f).tolist()]
    for x, s in zip(f, st):
        turn = (x / (2 * math.pi)) % 1.0
        d = abs(s / 2.0 ** 64 - turn)
        assert min(d, 1.0 - d) <= 2.0 ** -52, (x, s)
    assert st[3] == 0
    with pytest.raises(ola.OrthrosError):
        ola.orthros_rotary_steps([1.0, float("inf")])


P = 1 << 12  # a 16-byte aligned address that no refused call reads


def _rotate(lib, **o):
    a = dict(x=P, xs=256, pos=P, al=None, be=None, st=P, rot=64, lay=0, amp=1.0, n=2, H=4, d=64, dt=0, y=2 * P, ys=256)
    a.update(o)
    return lib.orthros_rotate(a["x"], a["xs"], a["pos"], a["al"], a["be"], a["st"], a["rot"], a["lay"], a["amp"], a["n"],
                              a["H"], a["d"], a["dt"], a["y"], a["ys"], None)


@pytest.mark.parametrize("over,code", [
    (dict(n=-1), 1), (dict(H=0), 1), (dict(dt=7), 1), (dict(d=96), 2), (dict(rot=0), 1), (dict(rot=66), 1),
    (dict(rot=63), 1), (dict(rot=40), 2), (dict(lay=2), 1), (dict(amp=float("nan")), 1), (dict(st=None), 1),
    (dict(st=P + 4), 1), (dict(al=P), 1), (dict(al=P, be=P + 4), 1), (dict(x=None), 1), (dict(x=P + 8), 1),
    (dict(xs=-8), 1), (dict(xs=260), 1), (dict(ys=248), 1), (dict(y=None), 1), (dict(y=P, xs=512), 1),
    (dict(pos=None), 1), (dict(H=1 << 20), 2)])
def test_rotate_refusals(lib, over, code):
    assert _rotate(lib, **over) == code
    assert ola.orthros_last_error() != ""


def _backward(lib, **o):
    a = dict(dy=P, dys=256, x=P, xs=256, pos=P, al=P, st=P, rot=64, lay=0, amp=1.0, n=2, H=4, d=64, dt=0, dx=2 * P,
             dxs=256, da=P, db=P, ws=P, wsb=1 << 24)
    a.update(o)
    return lib.orthros_rotate_backward(a["dy"], a["dys"], a["x"], a["xs"], a["pos"], a["al"], a["st"], a["rot"], a["lay"],
                                       a["amp"], a["n"], a["H"], a["d"], a["dt"], a["dx"], a["dxs"], a["da"], a["db"],
                                       a["ws"], a["wsb"], None)


@pytest.mark.parametrize("over,code", [
    (dict(n=-1), 1), (dict(d=32), 2), (dict(rot=24), 2), (dict(al=P + 4), 1), (dict(da=None), 1), (dict(ws=None), 4),
    (dict(wsb=64), 4), (dict(ws=P + 16), 1), (dict(dy=None), 1), (dict(x=None), 1), (dict(dxs=128), 1),
    (dict(dx=P, dxs=512), 1), (dict(pos=None), 1)])
def test_backward_refusals(lib, over, code):
    assert _backward(lib, **over) == code


def _append(lib, **o):
    a = dict(q=P, qs=256, qo=P, qos=256, k=P, ks=128, v=P, vs=128, ab=None, bb=None, ao=None, bo=None, st=P, rot=64,
             lay=0, amp=1.0, ts=P, tp=P, op=P, nn=2, no=1, Hq=4, Hkv=2, d=64, dt=0, qr=P, qor=P, kc=P, vc=P, bt=P, B=1,
             mp=4, ps=16, np_=4, ws=P, wsb=256)
    a.update(o)
    return lib.orthros_rotate_append(
        a["q"], a["qs"], a["qo"], a["qos"], a["k"], a["ks"], a["v"], a["vs"], a["ab"], a["bb"], a["ao"], a["bo"], a["st"],
        a["rot"], a["lay"], a["amp"], a["ts"], a["tp"], a["op"], a["nn"], a["no"], a["Hq"], a["Hkv"], a["d"], a["dt"],
        a["qr"], a["qor"], a["kc"], a["vc"], a["bt"], a["B"], a["mp"], a["ps"], a["np_"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("over,code", [
    (dict(nn=-1), 1), (dict(no=-1), 1), (dict(Hkv=0), 1), (dict(d=80), 2), (dict(dt=3), 1), (dict(rot=8), 2),
    (dict(st=None), 1), (dict(nn=0, st=None), 1), (dict(ab=P), 1), (dict(ao=P, bo=None), 1), (dict(ws=None), 4),
    (dict(wsb=8), 4), (dict(ws=P + 64), 1), (dict(k=None), 1), (dict(v=P + 4), 1), (dict(ks=4), 1), (dict(qr=None), 1),
    (dict(ts=None), 1), (dict(tp=None), 1), (dict(bt=None), 1), (dict(kc=None), 1), (dict(vc=P + 8), 1), (dict(B=0), 1),
    (dict(ps=0), 1), (dict(mp=0), 1), (dict(np_=0), 1), (dict(qo=None), 1), (dict(qor=None), 1), (dict(op=None), 1)])
def test_append_refusals(lib, over, code):
    assert _append(lib, **over) == code


def test_binding_refusals(lib):
    st = torch.zeros(32, dtype=torch.int64)
    x = torch.zeros(3, 4, 64)
    pos = torch.zeros(3, dtype=torch.int32)
    for bad in (dict(layout="other"), dict(alpha=torch.zeros(4, 32)), dict(alpha=torch.zeros(4, 64, dtype=torch.bfloat16)),
                dict(out=torch.zeros(3, 4, 64, dtype=torch.bfloat16)), dict(out=torch.zeros(2, 4, 64))):
        with pytest.raises(ola.OrthrosError):
            ola.orthros_rotate(x, pos, st, **bad)
    with pytest.raises(ola.OrthrosError):
        ola.orthros_rotate(x.transpose(1, 2).contiguous().transpose(1, 2), pos, st)  # heads not contiguous
    with pytest.raises(ola.OrthrosError):
        ola.orthros_rotate(x, pos.long(), st)
    with pytest.raises(ola.OrthrosError):
        ola.orthros_rotate(x, pos, st.float())


# ---------------------------------------------------------------------------
# GPU parity
# ---------------------------------------------------------------------------
SHAPES = [(1, 1, 64, 64), (1, 32, 128, 128), (17, 3, 64, 16), (33, 5, 128, 48), (130, 32, 128, 128), (515, 12, 128, 96),
          (64, 40, 64, 32), (7, 33, 128, 64)]


def make(n, H, d, dtype, seed, far=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, H, d, generator=g).to(dtype)
    al = 1.0 + 0.1 * torch.randn(H, d, generator=g)
    be = 0.1 * torch.randn(H, d, generator=g)
    pos = torch.randint(0, 200000, (n,), generator=g, dtype=torch.int32)
    if far and n > 4:
        pos[:4] = torch.tensor([0, -3, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    return x, al, be, pos


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n,H,d,rot", SHAPES)
def test_rotate(n, H, d, rot, dtype, layout):
    x, al, be, pos = make(n, H, d, dtype, seed=n + H)
    steps = ola.orthros_rotary_steps(frequencies(rot))
    amp = 1.25
    for affine in (False, True):
        u = x.double() * al.double() + be.double() if affine else x.double()
        mag_u = (x.double() * al.double()).abs() + be.double().abs() if affine else u.abs()
        ref, _ = plain_rotate(u, pos, steps, layout, amp)
        _, mag = plain_rotate(mag_u, pos, steps, layout, amp)
        kw = dict(alpha=al.cuda(), beta=be.cuda()) if affine else {}
        y = ola.orthros_rotate(x.cuda(), pos.cuda(), steps.cuda(), layout=layout, amplitude=amp, **kw)
        check(y, ref, mag, dtype, f"affine={affine}")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_rotate_strides_and_in_place(dtype):
    """Slices of a packed projection, one broadcast token, and y = x give the contiguous call's bits."""
    n, Hq, Hkv, d = 37, 6, 2, 64
    g = torch.Generator().manual_seed(3)
    packed = torch.randn(n, Hq + 2 * Hkv, d, generator=g).to(dtype).cuda()
    pos = torch.randint(0, 5000, (n,), generator=g, dtype=torch.int32).cuda()
    steps = ola.orthros_rotary_steps(frequencies(32)).cuda()
    want_q = ola.orthros_rotate(packed[:, :Hq].contiguous(), pos, steps)
    want_k = ola.orthros_rotate(packed[:, Hq:Hq + Hkv].contiguous(), pos, steps)
    before = packed.clone()
    assert torch.equal(ola.orthros_rotate(packed[:, :Hq], pos, steps), want_q)
    k = packed[:, Hq:Hq + Hkv]
    ola.orthros_rotate(k, pos, steps, out=k)
    assert torch.equal(packed[:, Hq:Hq + Hkv], want_k)
    assert torch.equal(packed[:, :Hq], before[:, :Hq]) and torch.equal(packed[:, Hq + Hkv:], before[:, Hq + Hkv:])
    one = before[:1, :Hq].expand(n, Hq, d)
    assert torch.equal(ola.orthros_rotate(one, pos, steps), ola.orthros_rotate(one.contiguous(), pos, steps))
    assert ola.orthros_rotate(packed[:0, :Hq], pos[:0], steps).shape == (0, Hq, d)


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n,H,d,rot", SHAPES + [(2100, 4, 64, 64)])
def test_backward(n, H, d, rot, dtype, layout):
    x, al, _, pos = make(n, H, d, dtype, seed=7 * n + H)
    dy = torch.randn(n, H, d, generator=torch.Generator().manual_seed(n)).to(dtype)
    steps = ola.orthros_rotary_steps(frequencies(rot))
    amp = 0.75
    g, mag = plain_rotate(dy.double(), pos, steps, layout, amp, sign=-1.0)
    args = (dy.cuda(), x.cuda(), pos.cuda(), steps.cuda())
    kw = dict(layout=layout, amplitude=amp, alpha=al.cuda())
    dx, da, db = ola.orthros_rotate_backward(*args, **kw)
    check(dx, g * al.double(), mag * al.double().abs(), dtype, "dx")
    for got, ref, terms in ((da, (g * x.double()).sum(0), mag * x.double().abs()), (db, g.sum(0), mag)):
        tol = ((n + 12) * 2.0 ** -24 + ANGLE) * terms.sum(0) + 1e-37
        assert bool(((got.double().cpu() - ref).abs() <= tol).all())
    # the same call gives the same bits; without the affine's gradient, the same dx
    dx2, da2, db2 = ola.orthros_rotate_backward(*args, **kw)
    assert torch.equal(dx, dx2) and torch.equal(da, da2) and torch.equal(db, db2)
    dx3, none, _ = ola.orthros_rotate_backward(args[0], None, *args[2:], affine_grads=False, **kw)
    assert none is None and torch.equal(dx, dx3)
    # no alpha: the transposed rotation alone
    dx4, _, _ = ola.orthros_rotate_backward(*args, layout=layout, amplitude=amp)
    check(dx4, g, mag, dtype, "dx without alpha")


@pytest.mark.gpu
def test_backward_against_differences():
    """Central differences of sum(w . y) along a random direction of x, alpha and beta (the map is
    linear in each, so the difference is exact up to fp32 rounding of y: 12 * 2^-24 per element)."""
    n, H, d, rot = 29, 3, 64, 48
    x, al, be, pos = make(n, H, d, torch.float32, seed=5)
    g = torch.Generator().manual_seed(6)
    w = torch.randn(n, H, d, generator=g)
    steps = ola.orthros_rotary_steps(frequencies(rot)).cuda()
    dx, da, db = ola.orthros_rotate_backward(w.cuda(), x.cuda(), pos.cuda(), steps, alpha=al.cuda())

    def loss(x_, al_, be_):
        y = ola.orthros_rotate(x_.cuda(), pos.cuda(), steps, alpha=al_.cuda(), beta=be_.cuda())
        return float((w.double() * y.double().cpu()).sum())

    noise = 2 * 12 * 2.0 ** -24 * float((w.abs() * 8).sum())  # |u_a| + |u_b| <= 8 here, both evaluations
    for name, base, grad in (("x", x, dx), ("alpha", al, da), ("beta", be, db)):
        e = torch.randn(base.shape, generator=g)
        args = {"x": x, "alpha": al, "beta": be}
        up, dn = dict(args, **{name: base + e}), dict(args, **{name: base - e})
        num = (loss(up["x"], up["alpha"], up["beta"]) - loss(dn["x"], dn["alpha"], dn["beta"])) / 2
        ana = float((grad.double().cpu() * e.double()).sum())
        assert abs(num - ana) <= noise, (name, num, ana, noise)


@pytest.mark.gpu
def test_backward_undoes_the_rotation():
    """m = 1: the gradient of the rotation applied to its output gives the input back."""
    x, _, _, pos = make(300, 8, 128, torch.float32, seed=8)
    steps = ola.orthros_rotary_steps(frequencies(128)).cuda()
    y = ola.orthros_rotate(x.cuda(), pos.cuda(), steps, layout="interleaved")
    back, _, _ = ola.orthros_rotate_backward(y, None, pos.cuda(), steps, layout="interleaved", affine_grads=False,
                                             out=(y, None, None))
    assert back.data_ptr() == y.data_ptr()
    assert float((back.cpu() - x).abs().max()) <= 2 * ANGLE * 2 * float(x.abs().max())


def make_append(dtype, B, new, hist, Hq, Hkv, d, page, seed):
    g = torch.Generator().manual_seed(seed)
    total = [a + b for a, b in zip(new, hist)]
    mp = max(1, max((t + page - 1) // page for t in total)) + 1
    pages = B * mp
    bt = torch.randperm(pages + 2, generator=g)[:pages].to(torch.int32).view(B, mp)
    kc = torch.randn(pages + 2, page, Hkv, d, generator=g).to(dtype)
    vc = torch.randn(pages + 2, page, Hkv, d, generator=g).to(dtype)
    seq = torch.tensor([b for b, n in enumerate(new) for _ in range(n)], dtype=torch.int32)
    pos = torch.tensor([h + i for n, h in zip(new, hist) for i in range(n)], dtype=torch.int32)
    n = len(seq)
    order = torch.randperm(n, generator=g)
    packed = torch.randn(n, Hq + 2 * Hkv, d, generator=g).to(dtype)
    return bt, kc, vc, seq[order], pos[order], packed


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("new,hist,Hq,Hkv,d,page,rot", [
    ([1], [0], 1, 1, 64, 1, 16), ([1, 1, 1], [0, 7, 300], 8, 2, 128, 64, 128), ([5, 0, 130, 1], [0, 3, 17, 64], 4, 4, 64, 16, 32),
    ([70, 33], [1000, 2], 32, 8, 128, 3, 96), ([2, 3, 4, 5, 6], [5, 4, 3, 2, 1], 6, 2, 64, 48, 64)])
def test_append(new, hist, Hq, Hkv, d, page, rot, dtype, layout):
    B = len(new)
    bt, kc, vc, seq, pos, packed = make_append(dtype, B, new, hist, Hq, Hkv, d, page, seed=sum(new) + page)
    n = len(seq)
    _, al, be, _ = make(1, Hq, d, dtype, seed=1)
    _, al2, be2, _ = make(1, Hq, d, dtype, seed=2)
    g = torch.Generator().manual_seed(9)
    n_out = 3
    q_out = torch.randn(n_out, Hq, d, generator=g).to(dtype)
    opos = torch.randint(0, 70000, (n_out,), generator=g, dtype=torch.int32)
    steps = ola.orthros_rotary_steps(frequencies(rot))
    amp = 1.1
    dev = packed.cuda()
    kg, vg = kc.cuda(), vc.cuda()
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    q, k, v = dev[:, :Hq], dev[:, Hq:Hq + Hkv], dev[:, Hq + Hkv:]
    qr, qor = ola.orthros_rotate_append(q, k, v, kg, vg, bt.cuda(), seq.cuda(), pos.cuda(), steps.cuda(), layout=layout,
                                        amplitude=amp, q_out=q_out.cuda(), out_positions=opos.cuda(),
                                        alpha_base=al.cuda(), beta_base=be.cuda(), alpha_out=al2.cuda(),
                                        beta_out=be2.cuda(), workspace=ws)
    assert ola.orthros_check(ws) == (0, 0)
    for got, raw, a, b, p in ((qr, packed[:, :Hq], al, be, pos), (qor, q_out, al2, be2, opos)):
        ref, _ = plain_rotate(raw.double() * a.double() + b.double(), p, steps, layout, amp)
        _, mag = plain_rotate((raw.double() * a.double()).abs() + b.double().abs(), p, steps, layout, amp)
        check(got, ref, mag, dtype, "queries")
    slots = bt[seq.long(), (pos // page).long()].long() * page + (pos % page).long()
    ref, mag = plain_rotate(packed[:, Hq:Hq + Hkv].double(), pos, steps, layout, amp)
    check(kg.flatten(0, 1)[slots.cuda()], ref, mag, dtype, "keys")
    vw, kw = vc.flatten(0, 1).clone(), kc.flatten(0, 1).clone()
    vw[slots] = packed[:, Hq + Hkv:]
    assert torch.equal(vg.flatten(0, 1).cpu(), vw)
    rest = torch.ones(len(kw), dtype=torch.bool)
    rest[slots] = False
    assert torch.equal(kg.flatten(0, 1).cpu()[rest], kw[rest])  # nothing else is touched
    # keys alone, and the output stream alone
    k2, v2 = kc.cuda(), vc.cuda()
    a, b = ola.orthros_rotate_append(None, k, v, k2, v2, bt.cuda(), seq.cuda(), pos.cuda(), steps.cuda(), layout=layout,
                                     amplitude=amp)
    assert a is None and b is None and torch.equal(k2, kg) and torch.equal(v2, vg)
    _, b = ola.orthros_rotate_append(None, k[:0], v[:0], k2, v2, bt.cuda(), seq.cuda()[:0], pos.cuda()[:0], steps.cuda(),
                                     layout=layout, amplitude=amp, q_out=q_out.cuda(), out_positions=opos.cuda(),
                                     alpha_out=al2.cuda(), beta_out=be2.cuda())
    assert torch.equal(b, qor) and torch.equal(k2, kg)


@pytest.mark.gpu
def test_append_flags_bad_data():
    """Sequences, positions and page ids outside their ranges: a status bit, that token's write skipped,
    every other token written."""
    new, hist = [3, 3, 3], [0, 0, 0]
    bt, kc, vc, _, _, packed = make_append(torch.bfloat16, 3, new, hist, 4, 2, 64, 4, seed=1)
    mp = bt.shape[1]
    steps = ola.orthros_rotary_steps(frequencies(64)).cuda()
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    k, v = packed[:, 4:6].cuda(), packed[:, 6:].cuda()
    good = [(b, i) for b in range(3) for i in range(3)]
    for where, value, bit in ((0, (3, 0), 1), (4, (-1, 2), 1), (8, (2, 4 * mp), 1), (2, (0, -1), 1), (5, (1, 2), 2)):
        rows = list(good)
        rows[where] = value
        table = bt.clone()
        if bit == 2:
            table[1, 0] = len(kc)  # past the pool: all three tokens of sequence 1
        seq = torch.tensor([r[0] for r in rows], dtype=torch.int32)
        pos = torch.tensor([r[1] for r in rows], dtype=torch.int32)
        kg, vg = kc.cuda(), vc.cuda()
        ola.orthros_rotate_append(None, k, v, kg, vg, table.cuda(), seq.cuda(), pos.cuda(), steps, workspace=ws)
        assert ola.orthros_check(ws) == (5, bit)
        keep = [i for i in range(9) if i != where] if bit == 1 else [0, 1, 2, 6, 7, 8]
        want = vc.flatten(0, 1).clone()
        for i in keep:
            want[int(bt[rows[i][0], 0]) * 4 + rows[i][1]] = packed[i, 6:]
        assert torch.equal(vg.flatten(0, 1).cpu(), want)


@pytest.mark.gpu
def test_graph_and_side_stream():
    """The three calls captured in a graph, and on a stream of the caller's, give the eager bits."""
    new, hist = [4, 9], [2, 60]
    bt, kc, vc, seq, pos, packed = make_append(torch.bfloat16, 2, new, hist, 8, 2, 128, 16, seed=2)
    _, al, be, _ = make(1, 8, 128, torch.float32, seed=1)
    steps = ola.orthros_rotary_steps(frequencies(128)).cuda()
    dev, al, be, bt, seq, pos = packed.cuda(), al.cuda(), be.cuda(), bt.cuda(), seq.cuda(), pos.cuda()
    kg, vg = kc.cuda(), vc.cuda()
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    ws2 = torch.empty(ola.orthros_rotate_backward_workspace_size(13, 8, 128), dtype=torch.uint8, device="cuda")
    q = dev[:, :8]

    def step():
        y = ola.orthros_rotate(q, pos, steps, alpha=al, beta=be)
        g = ola.orthros_rotate_backward(y, q, pos, steps, alpha=al, workspace=ws2)
        r, _ = ola.orthros_rotate_append(q, dev[:, 8:10], dev[:, 10:], kg, vg, bt, seq, pos, steps, alpha_base=al,
                                         beta_base=be, workspace=ws)
        return (y, *g, r)

    want = [t.clone() for t in step()] + [kg.clone(), vg.clone()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        kg.copy_(kc)
        got = list(step()) + [kg, vg]
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for t in out:
        t.zero_()
    kg.copy_(kc.cuda())
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(list(out) + [kg, vg], want))


@pytest.mark.gpu
@pytest.mark.parametrize("handle", [False, True])
def test_stream_argument_owns_what_the_call_allocates(handle):
    """Outputs of a call on another stream are not taken from memory that the current stream still writes."""
    bt, kc, vc, seq, pos, packed = make_append(torch.bfloat16, 2, [4, 9], [2, 60], 8, 2, 128, 16, seed=2)
    _, al, be, _ = make(1, 8, 128, torch.float32, seed=1)
    steps = ola.orthros_rotary_steps(frequencies(128)).cuda()
    dev, al, be, bt, seq, pos = packed.cuda(), al.cuda(), be.cuda(), bt.cuda(), seq.cuda(), pos.cuda()
    kg, vg = kc.cuda(), vc.cuda()
    q = dev[:, :8]
    dy = torch.ones_like(q)

    def step(**kw):
        return (ola.orthros_rotate(q, pos, steps, alpha=al, beta=be, **kw),
                *ola.orthros_rotate_backward(dy, q, pos, steps, alpha=al, **kw),
                ola.orthros_rotate_append(q, dev[:, 8:10], dev[:, 10:], kg, vg, bt, seq, pos, steps, alpha_base=al,
                                          beta_base=be, **kw)[0])

    want = [t.clone() for t in step()]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # the current stream is behind, with writes to what it has freed
    stale = [torch.empty_like(t) for t in want for _ in range(3)]
    for t in stale:
        t.fill_(float("nan"))
    del t, stale
    got = step(stream=s.cuda_stream if handle else s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


# ---------------------------------------------------------------------------
# steps and far positions against the angle itself
# ---------------------------------------------------------------------------
def inverse_two_pi(bits=400):
    """floor(2^bits / 2 pi), from Machin's formula pi = 16 arctan(1/5) - 4 arctan(1/239) in integers."""
    one = 1 << (bits + 64)

    def arctan_of_one_over(n):
        total, term, k = 0, one // n, 0
        while term:
            total += term // (2 * k + 1) * (-1) ** k
            term //= n * n
            k += 1
        return total

    pi = 16 * arctan_of_one_over(5) - 4 * arctan_of_one_over(239)
    return (one << bits) // (2 * pi)


def turn_units(x):
    """x / 2 pi modulo a turn, in 2^-64 turns, as a Fraction (x a double or a Fraction)."""
    from fractions import Fraction

    return Fraction(x) * inverse_two_pi() / (1 << 400) % 1 * (1 << 64)


def test_steps_are_the_nearest_units(lib):
    """A step is the frequency's fraction of a turn rounded to 2^-64 turn, not to a double's 53 bits: at
    position 2^31 the angle is off by 2^-34 turn (4e-10 rad) at most."""
    freq = [1.0, 0.5, 1e-3, 2 * math.pi, -1.0, 2 * math.pi + 1.0, 3.0, 1e-12, -1e-30, 1e-25, 1e6, 123456.789, 2.0 ** 40]
    for rule in (dict(), dict(scaling="bands", factor=8.0, original_length=8192.0)):
        freq += ola.orthros_rotary_frequencies(128, 500000.0, **rule)[0].tolist()
    steps = [int(s) % 2 ** 64 for s in ola.orthros_rotary_steps(freq).tolist()]
    for f, s in zip(freq, steps):
        off = (s - turn_units(f)) % (1 << 64)
        assert min(off, (1 << 64) - off) <= 0.5 + 2.0 ** -20, (f, s)
    # far outside any use: still a defined step, no overflow
    ola.orthros_rotary_steps([1e300, -1e300, 1.7e308, 5e-324, -5e-324])


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_far_positions_against_the_angle(layout):
    """fp32 at the ends of the 32-bit positions, against position times frequency in 400 bits."""
    rot, H, d = 64, 2, 64
    freq = frequencies(rot)
    pos = [0, 1, -1, 131071, 10 ** 6 + 1, 2 ** 29 + 3, 2 ** 30 + 7, 2 ** 31 - 1, -2 ** 31, -2 ** 31 + 1, 1999999973]
    x = torch.randn(len(pos), H, d, generator=torch.Generator().manual_seed(4))
    from fractions import Fraction

    ph = torch.tensor([[float(turn_units(Fraction(f) * t)) / 2.0 ** 64 for f in freq.tolist()] for t in pos],
                      dtype=torch.float64)
    c, s = torch.cos(2 * math.pi * ph)[:, None], torch.sin(2 * math.pi * ph)[:, None]
    ia, ib = channels(rot, layout)
    u, ref, mag = x.double(), x.double(), x.double().abs()
    ref[..., ia], ref[..., ib] = u[..., ia] * c - u[..., ib] * s, u[..., ia] * s + u[..., ib] * c
    m = mag[..., ia] + mag[..., ib]
    mag[..., ia], mag[..., ib] = m, m
    y = ola.orthros_rotate(x.cuda(), torch.tensor(pos, dtype=torch.int32).cuda(), ola.orthros_rotary_steps(freq).cuda(),
                           layout=layout)
    check(y, ref, mag, torch.float32, "far positions")


# ---------------------------------------------------------------------------
# blocks that walk many tables of angles: with few heads a block has many tokens
# side by side, with many heads few; either way more than 128 tokens (a run of
# looked-up positions and page slots) here, and odd rests
# ---------------------------------------------------------------------------
def long_angles(pos, steps):
    """cos, sin [n, pairs] in fp64 on the GPU: int64 products wrap as the phase does."""
    ph = (pos.long()[:, None] * steps[None, :]).double() * 2.0 ** -64
    return torch.cos(2 * math.pi * ph), torch.sin(2 * math.pi * ph)


def long_rotate(u, mag, pos, steps, layout, amp, sign=1.0):
    """plain_rotate on the GPU, with the magnitudes given."""
    c, s = long_angles(pos, steps)
    c, s = amp * c[:, None, :], amp * sign * s[:, None, :]
    ia, ib = channels(2 * steps.numel(), layout)
    y, m = u.clone(), mag.clone()
    y[..., ia] = u[..., ia] * c - u[..., ib] * s
    y[..., ib] = u[..., ia] * s + u[..., ib] * c
    m[..., ia] = m[..., ib] = amp * (mag[..., ia] + mag[..., ib])
    return y, m


def long_check(got, raw, affine, pos, steps, layout, amp, what, sign=1.0):
    for i in range(0, got.shape[0], 8192):
        r = slice(i, i + 8192)
        u = raw[r].double()
        mag = u.abs()
        if affine is not None:
            al, be = affine[0].double(), affine[1].double()
            mag = mag * al.abs() + be.abs()
            u = u * al + be
        ref, m = long_rotate(u, mag, pos[r], steps, layout, amp, sign)
        tol = HALF_STEP[got.dtype] * ref.abs() + ANGLE * m + 1e-37
        err = (got[r].double() - ref).abs() / tol
        assert float(err.max()) <= 1, f"{what}, tokens from {i}: {float(err.max()):.3f} of the tolerance"


def long_inputs(n, H, d, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")
    pos = torch.randint(0, 200000, (n,), generator=g, device="cuda", dtype=torch.int32)
    return rn(n, H, d).to(dtype), 1.0 + 0.1 * rn(H, d), 0.1 * rn(H, d), pos, rn(n, H, d).to(dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("n,H,d,rot,dtype", [
    (200001, 1, 64, 64, torch.bfloat16), (45001, 5, 128, 48, torch.bfloat16), (45001, 32, 128, 128, torch.bfloat16),
    (100001, 1, 64, 32, torch.float32), (25001, 32, 128, 128, torch.float32)])
def test_rotate_long(n, H, d, rot, dtype, layout):
    x, al, be, pos, _ = long_inputs(n, H, d, dtype, seed=H)
    steps = ola.orthros_rotary_steps(frequencies(rot)).cuda()
    y = ola.orthros_rotate(x, pos, steps, layout=layout, amplitude=1.25, alpha=al, beta=be)
    long_check(y, x, (al, be), pos, steps, layout, 1.25, "rotate")


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("n,H,d,rot,dtype", [
    (24001, 2, 64, 64, torch.bfloat16), (24001, 32, 128, 128, torch.bfloat16), (21001, 8, 128, 96, torch.float32),
    (24001, 40, 64, 16, torch.float32)])
def test_backward_long(n, H, d, rot, dtype, layout):
    x, al, _, pos, dy = long_inputs(n, H, d, dtype, seed=3 * H)
    steps = ola.orthros_rotary_steps(frequencies(rot)).cuda()
    dx, da, db = ola.orthros_rotate_backward(dy, x, pos, steps, layout=layout, amplitude=0.75, alpha=al)
    sums = [torch.zeros(H, d, dtype=torch.float64, device="cuda") for _ in range(4)]
    for i in range(0, n, 8192):
        r = slice(i, i + 8192)
        g, m = long_rotate(dy[r].double(), dy[r].double().abs(), pos[r], steps, layout, 0.75, -1.0)
        err = (dx[r].double() - g * al.double()).abs() / (HALF_STEP[dtype] * (g * al).abs() + ANGLE * m * al.abs() + 1e-37)
        assert float(err.max()) <= 1, f"dx, tokens from {i}: {float(err.max()):.3f} of the tolerance"
        for to, v in zip(sums, ((g * x[r].double()), g, m * x[r].double().abs(), m)):
            to += v.sum(0)
    # additions in a row: a block's tokens, its token lanes (16 at most), the blocks' partials
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    depth = 2 * ((n + sms - 1) // sms + 16 + sms)  # (twice: groups of heads share the SMs)
    for got, ref, terms in ((da, sums[0], sums[2]), (db, sums[1], sums[3])):
        assert bool(((got.double() - ref).abs() <= ((depth + 12) * 2.0 ** -24 + ANGLE) * terms).all())
    dx2, none, _ = ola.orthros_rotate_backward(dy, None, pos, steps, layout=layout, amplitude=0.75, alpha=al, affine_grads=False)
    assert none is None and torch.equal(dx, dx2)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("new,n_out,Hq,Hkv,d,page,rot,layout", [
    ([9000, 1, 4000, 7001], 9001, 32, 8, 128, 16, 128, "half"), ([70001], 3, 1, 1, 64, 7, 32, "interleaved")])
def test_append_long(new, n_out, Hq, Hkv, d, page, rot, layout, dtype):
    B, n = len(new), sum(new)
    packed, al, be, _, _ = long_inputs(n, Hq + 2 * Hkv, d, dtype, seed=n)
    q_out, al2, be2, opos, _ = long_inputs(n_out, Hq, d, dtype, seed=n + 1)
    al, be = al[:Hq].contiguous(), be[:Hq].contiguous()
    g = torch.Generator().manual_seed(n)
    mp = max((m + 50 + page - 1) // page for m in new)
    bt = torch.randperm(B * mp, generator=g).to(torch.int32).view(B, mp).cuda()
    seq = torch.cat([torch.full((m,), b, dtype=torch.int32) for b, m in enumerate(new)]).cuda()
    pos = torch.cat([torch.arange(7 * b, 7 * b + m, dtype=torch.int32) for b, m in enumerate(new)]).cuda()
    kc = torch.full((B * mp, page, Hkv, d), 7.0, dtype=dtype, device="cuda")
    vc = torch.full_like(kc, 9.0)
    steps = ola.orthros_rotary_steps(frequencies(rot)).cuda()
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    q, k, v = packed[:, :Hq], packed[:, Hq:Hq + Hkv], packed[:, Hq + Hkv:]
    qr, qor = ola.orthros_rotate_append(q, k, v, kc, vc, bt, seq, pos, steps, layout=layout, amplitude=1.1, q_out=q_out,
                                        out_positions=opos, alpha_base=al, beta_base=be, alpha_out=al2, beta_out=be2,
                                        workspace=ws)
    assert ola.orthros_check(ws) == (0, 0)
    slots = bt[seq.long(), torch.div(pos, page, rounding_mode="floor").long()].long() * page + (pos % page).long()
    long_check(qr, q, (al, be), pos, steps, layout, 1.1, "queries")
    long_check(qor, q_out, (al2, be2), opos, steps, layout, 1.1, "output queries")
    long_check(kc.flatten(0, 1)[slots], k, None, pos, steps, layout, 1.1, "keys")
    assert torch.equal(vc.flatten(0, 1)[slots], v)
    rest = torch.ones(B * mp * page, dtype=torch.bool, device="cuda")
    rest[slots] = False
    assert bool((kc.flatten(0, 1)[rest] == 7).all()) and bool((vc.flatten(0, 1)[rest] == 9).all())
