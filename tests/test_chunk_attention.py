"""orthros_chunk_attention (new tokens over a paged cache that holds their keys)
against softmax attention in fp64.

Tolerances, with S = max_j scale sum_c |q_c k_jc| of a row and A = sum_j p_j |v_j| / l:
logits are 128 products accumulated in fp32, off by at most 128 * 2^-24 S; one
exponential in 64 comes from a cubic that is off by 7.5e-5, the rest from
ex2.approx (2^-22). So |lse| is off by at most 2^-17 S + 8e-5 + 2^-20 |lse| (sum, log,
product with scale), and o by the same relative error of every weight and of the
sum (2 (2^-17 S + 8e-5) A), by P's rounding to bf16 (half a step: 2^-8 A) and by its
own (2^-8 |o|).

The cubic is gone from the kernel: every exponential is ex2.approx, so 8e-5 is wider than
it need be. check_fp32 below has the bound of the present code, and its tests hold the sums
and weights to it.
"""
import numpy as np
import pytest
import torch

import efficient_long_context_gb300 as ola


@pytest.fixture(scope="module")
def lib():
    from efficient_long_context_gb300 import build

    build.build()
    return ola.load_library()


P = 1 << 12


def _call(lib, **o):
    a = dict(q=P, qi=P, kl=P, kc=P, vc=P, bt=P, B=2, n=3, mn=2, Hq=4, Hkv=2, d=64, w=8, sc=0.1, dt=0, mp=4, ps=16, np_=8,
             o=P, lse=P, ws=P, wsb=1 << 30)
    a.update(o)
    return lib.orthros_chunk_attention(a["q"], a["qi"], a["kl"], a["kc"], a["vc"], a["bt"], a["B"], a["n"], a["mn"], a["Hq"],
                                       a["Hkv"], a["d"], a["w"], a["sc"], a["dt"], a["mp"], a["ps"], a["np_"], a["o"],
                                       a["lse"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("over,code", [
    (dict(B=-1), 1), (dict(n=-1), 1), (dict(B=0), 1), (dict(mn=0), 1), (dict(Hq=3), 1), (dict(Hkv=0), 1), (dict(d=96), 2),
    (dict(dt=1), 2), (dict(dt=9), 1), (dict(Hq=258, Hkv=2), 2), (dict(w=0), 1), (dict(sc=0.0), 1), (dict(sc=-1.0), 1),
    (dict(sc=float("nan")), 1), (dict(sc=float("inf")), 1), (dict(mp=0), 1), (dict(ps=0), 1), (dict(np_=0), 1),
    (dict(np_=1 << 28), 2), (dict(mp=1 << 28), 2), (dict(ws=None), 4), (dict(wsb=1024), 4), (dict(ws=P + 16), 1),
    (dict(q=None), 1), (dict(o=None), 1), (dict(kc=None), 1), (dict(vc=None), 1), (dict(qi=None), 1), (dict(kl=None), 1),
    (dict(bt=None), 1), (dict(q=P + 8), 1), (dict(o=P + 8), 1), (dict(kc=P + 4), 1)])
def test_refusals(lib, over, code):
    assert _call(lib, **over) == code
    assert ola.orthros_last_error() != ""


def test_workspace_size(lib):
    f = ola.orthros_chunk_attention_workspace_size
    assert f(32, 32, 1, 32, 8, 128, 512, 64) > 0
    assert f(32, 32, 1, 32, 8, 128, 512, 64) < f(32, 3200, 100, 32, 8, 128, 512, 64)
    assert f(1, 100000, 100000, 32, 8, 128, 4096, 64) < 200 << 20  # partials do not grow with the tokens
    assert f(0, 0, 0, 4, 2, 64, 1, 64) > 0
    for bad in ((1, 4, 0, 4, 2, 64, 1, 64), (1, 4, 4, 4, 3, 64, 1, 64), (1, 4, 4, 4, 2, 32, 1, 64), (1, 4, 4, 4, 2, 64, 0, 64),
                (0, 4, 4, 4, 2, 64, 1, 64)):
        assert f(*bad) == 0
    assert f(1, 4, 4, 4, 2, 64, 1, 64, torch.float32) == 0


# ---------------------------------------------------------------------------
# GPU parity
# ---------------------------------------------------------------------------
def make(new, total, Hq, Hkv, d, page, window, seed, spare=3, fill=float("nan"), qscale=1.5):
    """A batch whose pages hold `fill` wherever no token of the batch looks."""
    g = torch.Generator().manual_seed(seed)
    B = len(new)
    mp = max(1, max((t + page - 1) // page for t in total))
    need = [(t + page - 1) // page for t in total]
    pool = sum(need) + spare
    perm = torch.randperm(pool, generator=g)
    bt = torch.full((B, mp), pool + 7, dtype=torch.int32)  # entries nobody may follow
    kc = torch.full((pool, page, Hkv, d), fill)
    vc = torch.full((pool, page, Hkv, d), fill)
    off = torch.randn(Hkv, d, generator=g) * 0.5
    K, V = [], []
    o = 0
    for b in range(B):
        k = torch.randn(total[b], Hkv, d, generator=g) + off
        v = torch.randn(total[b], Hkv, d, generator=g)
        K.append(k.bfloat16())
        V.append(v.bfloat16())
        first = max(0, total[b] - new[b] - window + 1) if new[b] else total[b]
        for i in range(need[b]):
            pg = int(perm[o + i])
            lo, hi = max(i * page, first), min(total[b], (i + 1) * page)
            if lo < hi:
                bt[b, i] = pg
                kc[pg, lo - i * page:hi - i * page] = K[b][lo:hi].float()
                vc[pg, lo - i * page:hi - i * page] = V[b][lo:hi].float()
        o += need[b]
    n = sum(new)
    q = (torch.randn(n, Hq, d, generator=g) * qscale).bfloat16()
    indptr = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32)
    return dict(q=q, K=K, V=V, kc=kc.bfloat16(), vc=vc.bfloat16(), bt=bt, indptr=indptr,
                lens=torch.tensor(total, dtype=torch.int32), new=new, total=total, window=window)


def plain(w, scale, rows=None):
    """fp64 (o, lse, A, S) of the batch's rows, computed on the GPU in fp64."""
    q = w["q"].cuda().double()
    n, Hq, d = q.shape
    out = [torch.empty(n, Hq, d, dtype=torch.float64, device="cuda"), torch.empty(n, Hq, dtype=torch.float64, device="cuda"),
           torch.empty(n, Hq, d, dtype=torch.float64, device="cuda"), torch.empty(n, Hq, dtype=torch.float64, device="cuda")]
    i0 = 0
    for b, (nb, L) in enumerate(zip(w["new"], w["total"])):
        if nb == 0:
            continue
        K, V = w["K"][b].cuda().double(), w["V"][b].cuda().double()
        g = Hq // K.shape[1]
        t = torch.arange(L - nb, L, device="cuda")[:, None]
        j = torch.arange(L, device="cuda")[None, :]
        seen = (j <= t) & (j > t - w["window"])
        for h in range(Hq):
            qq, kk, vv = q[i0:i0 + nb, h], K[:, h // g], V[:, h // g]
            z = (qq @ kk.T * scale).masked_fill(~seen, float("-inf"))
            p = torch.softmax(z, -1)
            out[0][i0:i0 + nb, h] = p @ vv
            out[1][i0:i0 + nb, h] = torch.logsumexp(z, -1)
            out[2][i0:i0 + nb, h] = p @ vv.abs()
            out[3][i0:i0 + nb, h] = (qq.abs() @ kk.abs().T * scale).masked_fill(~seen, 0).amax(-1)
        i0 += nb
    return out


def check(got, ref, what=""):
    o, lse = got[0].double(), got[1].double()
    ro, rl, A, S = ref
    weight = 2.0 ** -17 * S + 8e-5
    tol_l = weight + 2.0 ** -20 * rl.abs()
    tol_o = 2.0 ** -8 * ro.abs() + (2.0 ** -8 + 2 * weight[..., None]) * A + 1e-30
    assert bool(torch.isfinite(o).all()) and bool(torch.isfinite(lse).all()), f"{what}: not finite"
    el, eo = ((lse - rl).abs() / tol_l).max(), ((o - ro).abs() / tol_o).max()
    assert float(el) <= 1 and float(eo) <= 1, f"{what}: lse {float(el):.3f}, o {float(eo):.3f} of the tolerance"


def call(w, scale=None, **kw):
    return ola.orthros_chunk_attention(w["q"].cuda(), w["indptr"].cuda(), w["lens"].cuda(), w["kc"].cuda(), w["vc"].cuda(),
                                       w["bt"].cuda(), w["window"], scale, **kw)


CASES = [
    # new, total, Hq, Hkv, d, page, window
    ([1], [1], 1, 1, 64, 64, 1 << 20),
    ([1], [1], 32, 8, 128, 64, 1),
    ([1], [129], 4, 2, 128, 64, 1 << 20),
    ([1], [5000], 32, 8, 128, 64, 1 << 20),
    ([1, 1, 1], [1, 700, 128], 8, 2, 128, 16, 1 << 20),
    ([1, 1, 1, 1], [300, 2, 4097, 1000], 16, 16, 64, 128, 256),
    ([3], [3], 4, 4, 64, 8, 1 << 20),
    ([128], [128], 1, 1, 128, 64, 1 << 20),
    ([129], [129], 2, 2, 128, 64, 1 << 20),
    ([257], [1000], 1, 1, 64, 32, 100),
    ([33], [33], 8, 2, 128, 48, 2),
    ([70], [200], 32, 8, 128, 16, 127),
    ([65, 0, 1, 31, 64], [65, 9, 400, 31, 777], 8, 2, 128, 24, 128),
    ([300, 17], [5300, 17], 32, 8, 128, 64, 129),
    ([300, 17], [5300, 17], 32, 8, 64, 64, 1 << 20),
    ([700], [700], 16, 16, 128, 64, 512),
    ([1000, 1, 500], [9000, 6000, 500], 12, 4, 128, 64, 4096),
    ([40, 1, 3], [45, 260, 1003], 12, 1, 64, 16, 1 << 20),
    ([9, 1], [500, 300], 40, 1, 128, 64, 1 << 20),
    ([3, 2], [130, 5], 128, 1, 64, 8, 1 << 20),
    ([5, 1], [400, 40], 3, 1, 64, 8, 77),
    # kv heads that share no or a small factor with the number of SMs
    ([40, 1, 300], [900, 2000, 300], 10, 5, 128, 64, 1 << 20),
    ([7, 129], [300, 700], 24, 12, 64, 16, 200),
    ([1, 1], [777, 3000], 7, 7, 128, 64, 1 << 20),
    # page sizes without a copy box
    ([1, 1], [300, 7], 8, 2, 128, 1, 1 << 20),
    ([60, 1], [300, 129], 8, 2, 128, 5, 1 << 20),
    ([200], [900], 4, 4, 64, 12, 130),
]


@pytest.mark.gpu
@pytest.mark.parametrize("new,total,Hq,Hkv,d,page,window", CASES,
                         ids=lambda v: "-".join(map(str, v)) if isinstance(v, list) else str(v))
def test_parity(new, total, Hq, Hkv, d, page, window):
    w = make(new, total, Hq, Hkv, d, page, window, seed=sum(total) + page)
    ws = torch.empty(ola.orthros_chunk_attention_workspace_size(len(new), sum(new), max(new), Hq, Hkv, d, w["bt"].shape[1],
                                                                page), dtype=torch.uint8, device="cuda")
    got = call(w, max_new=max(new), workspace=ws)
    assert ola.orthros_check(ws) == (0, 0)
    check(got, plain(w, d ** -0.5))
    # the same call gives the same bits, whatever bound of the new tokens it is given
    again = call(w)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,d", [(32, 8, 128), (16, 16, 64)])
def test_many_sequences(Hq, Hkv, d):
    """More sequences than the plan's block has threads, one token or a few each, some none."""
    rng = np.random.default_rng(1)
    new = [int(x) for x in rng.choice([0, 1, 1, 2, 5], 1100)]
    total = [n + int(h) for n, h in zip(new, rng.integers(0, 40, 1100))]
    w = make(new, total, Hq, Hkv, d, 16, 20, seed=4)
    check(call(w, max_new=5), plain(w, d ** -0.5))


@pytest.mark.gpu
def test_long_history_and_large_logits():
    """One token over 40000 keys; logits in the hundreds, whose maxima keep moving."""
    for qs in (1.0, 60.0):
        w = make([1], [40000], 8, 2, 128, 64, 1 << 20, seed=6, qscale=qs)
        check(call(w), plain(w, 128 ** -0.5), f"q scale {qs}")
    w = make([130], [2000], 8, 2, 128, 64, 1 << 20, seed=7, qscale=60.0)
    check(call(w), plain(w, 128 ** -0.5))
    w = make([20], [700], 8, 2, 64, 64, 1 << 20, seed=8)
    check(call(w, 0.7), plain(w, 0.7), "scale 0.7")
    o, lse = ola.orthros_chunk_attention(w["q"].cuda(), w["indptr"].cuda(), w["lens"].cuda(), w["kc"].cuda(), w["vc"].cuda(),
                                         w["bt"].cuda(), w["window"], 0.7, out=(torch.empty_like(w["q"].cuda()), None))
    assert lse is None and torch.equal(o, call(w, 0.7)[0])


@pytest.mark.gpu
def test_largest_window():
    """A window of INT_MAX is every key (no index of the window's start may wrap)."""
    for new, total, Hq, Hkv in (([200, 1], [200, 130], 1, 1), ([70], [900], 8, 2)):
        w = make(new, total, Hq, Hkv, 64, 16, 1 << 20, seed=13)
        got = call(dict(w, window=2 ** 31 - 1))
        want = call(w)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.gpu
def test_pool_past_32_bit_offsets():
    """Pages whose elements lie past 2^31 of the pool."""
    page, Hkv, d = 64, 8, 128
    pool = (1 << 31) // (page * Hkv * d) + 200
    w = make([1, 40], [500, 900], 32, Hkv, d, page, 1 << 20, seed=9)
    small = w["kc"].shape[0]
    kc = torch.empty((pool, page, Hkv, d), dtype=torch.bfloat16, device="cuda")
    vc = torch.empty((pool, page, Hkv, d), dtype=torch.bfloat16, device="cuda")
    kc[pool - small:] = w["kc"].cuda()
    vc[pool - small:] = w["vc"].cuda()
    bt = torch.where(w["bt"] < small, w["bt"] + (pool - small), w["bt"])
    got = ola.orthros_chunk_attention(w["q"].cuda(), w["indptr"].cuda(), w["lens"].cuda(), kc, vc, bt.cuda(), w["window"])
    check(got, plain(w, d ** -0.5))


@pytest.mark.gpu
@pytest.mark.parametrize("m", [70, 40])  # with and without a plan kernel (64 tokens are one unit here)
def test_bad_lengths_and_pages(m):
    """Impossible data set their status bit and give NaN for the rows they concern, no others."""
    new, total = [2, m, 1], [300, 400, 90]
    w = make(new, total, 8, 2, 64, 16, 1 << 20, seed=10)
    ref = plain(w, 0.125)
    rows = [slice(0, 2), slice(2, 2 + m), slice(2 + m, 3 + m)]
    bound = m if m <= 64 else 3 + m
    ws = torch.empty(ola.orthros_chunk_attention_workspace_size(3, 3 + m, 3 + m, 8, 2, 64, w["bt"].shape[1], 16),
                     dtype=torch.uint8, device="cuda")

    def expect(bad, bits, **kw):
        v = dict(w, **kw)
        o, lse = call(v, workspace=ws, max_new=kw.get("max_new", bound))
        assert ola.orthros_check(ws) == (5, bits)
        for b in range(3):
            if b in bad:
                assert bool(torch.isnan(o[rows[b]]).all()) and bool(torch.isnan(lse[rows[b]]).all())
            else:
                check((o[rows[b]], lse[rows[b]]), [r[rows[b]] for r in ref])

    lens = lambda *v: torch.tensor(v, dtype=torch.int32)
    expect([0], 4, lens=lens(1, 400, 90))                           # fewer cached tokens than new ones
    expect([2], 4, lens=lens(300, 400, -5))
    expect([1], 4, lens=lens(300, w["bt"].shape[1] * 16 + 1, 90))   # past the block table
    expect([1], 4, max_new=m - 1)
    expect([0, 2], 4, lens=lens(1, 400, 0))
    expect([0, 1, 2], 4, lens=lens(1, 5, 0))
    bt = w["bt"].clone()
    bt[2, 0] = -1
    expect([2], 2, bt=bt)
    for indptr in ([0, 2, 2 + m, 2 + m], [1, 2, 2 + m, 3 + m], [0, 2 + m, 2, 3 + m], [0, 2, 2 + m, 4 + m]):
        expect([0, 1, 2], 4, indptr=lens(*indptr))
    # a single sequence, its units listed by the CTAs
    v = make([50], [60], 8, 2, 64, 16, 1 << 20, seed=14)
    for bad in (dict(lens=lens(49)), dict(indptr=lens(0, 49)), dict(lens=lens(1 << 20))):
        o, lse = call(dict(v, **bad), workspace=ws)
        assert ola.orthros_check(ws) == (5, 4)
        assert bool(torch.isnan(o).all()) and bool(torch.isnan(lse).all())
    check(call(v, workspace=ws), plain(v, 0.125))
    assert ola.orthros_check(ws) == (0, 0)
    # a bad page (keys 144 .. 159) in the middle of a chunk's keys: rows that stop before them are untouched
    v = make([256], [256], 1, 1, 64, 16, 1 << 20, seed=11)
    ref = plain(v, 0.125)
    bt = v["bt"].clone()
    bt[0, 9] = 1 << 20
    o, lse = call(dict(v, bt=bt))
    check((o[:144], lse[:144]), [r[:144] for r in ref])
    assert bool(torch.isnan(o[144:]).all()) and bool(torch.isnan(lse[144:]).all())
    # with a window, rows past it too; the same on pages that are gathered row by row
    for page, entry in ((16, 9), (12, 12)):
        v = make([256], [256], 1, 1, 128, page, 50, seed=17)
        ref = plain(v, 128 ** -0.5)
        bt = v["bt"].clone()
        bt[0, entry] = -7
        o, lse = call(dict(v, bt=bt))
        last = entry * page + page - 1 + 49  # the last row whose window holds one of its keys
        for rows in (slice(0, 144), slice(last + 1, 256)):
            check((o[rows], lse[rows]), [r[rows] for r in ref])
        assert bool(torch.isnan(o[144:last + 1]).all()) and bool(torch.isnan(lse[144:last + 1]).all())


@pytest.mark.gpu
def test_outputs_on_16_byte_boundaries():
    """o may start at any 16-byte boundary (32-byte stores only where they fit), and nothing beside it is touched."""
    for new, total in (([1, 40], [400, 500]), ([200], [300])):
        w = make(new, total, 8, 2, 128, 16, 1 << 20, seed=15)
        n = sum(new)
        flat = torch.full((n * 8 * 128 + 16,), 7.0, dtype=torch.bfloat16, device="cuda")
        o = flat[8:8 + n * 8 * 128].view(n, 8, 128)
        lse = torch.empty((n, 8), device="cuda")
        call(w, out=(o, lse))
        want = call(w)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
        assert bool((flat[:8] == 7).all()) and bool((flat[-8:] == 7).all())


@pytest.mark.gpu
def test_non_finite_query_stays_in_its_row():
    w = make([40, 3], [200, 50], 8, 2, 64, 16, 1 << 20, seed=16)
    want = call(w)
    q = w["q"].clone()
    q[5, 3] = float("nan")
    q[41, 0, 7] = float("inf")
    o, lse = call(dict(w, q=q))
    keep = torch.ones(43, 8, dtype=torch.bool)
    keep[5, 3] = keep[41, 0] = False
    assert torch.equal(o[keep.cuda()], want[0][keep.cuda()]) and torch.equal(lse[keep.cuda()], want[1][keep.cuda()])
    assert bool(torch.isnan(o[5, 3]).all()) and not bool(torch.isfinite(o[41, 0]).any())


@pytest.mark.gpu
def test_empty_calls():
    w = make([0, 0], [5, 9], 4, 2, 64, 16, 8, seed=1)
    o, lse = call(w)
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)


@pytest.mark.gpu
def test_graph_replays_growing_lengths_and_side_stream():
    """A captured step reads its lengths on the device: replayed with longer ones it follows them."""
    w = make([1, 30], [1000, 700], 8, 2, 128, 64, 1 << 20, seed=12)
    t = {k: w[k].cuda() for k in ("q", "indptr", "lens", "kc", "vc", "bt")}
    ws = torch.empty(ola.orthros_chunk_attention_workspace_size(2, 31, 30, 8, 2, 128, w["bt"].shape[1], 64),
                     dtype=torch.uint8, device="cuda")

    def step():
        return ola.orthros_chunk_attention(t["q"], t["indptr"], t["lens"], t["kc"], t["vc"], t["bt"], 1 << 20, max_new=30,
                                           workspace=ws)

    t["lens"].copy_(torch.tensor([300, 40]))
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for lens in ([300, 40], [999, 333], [1000, 700]):
        t["lens"].copy_(torch.tensor(lens))
        graph.replay()
        v = dict(w, total=lens, K=[k[:n] for k, n in zip(w["K"], lens)], V=[x[:n] for x, n in zip(w["V"], lens)])
        check(out, plain(v, 128 ** -0.5), str(lens))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        side = step()
    s.synchronize()
    assert torch.equal(side[0], out[0]) and torch.equal(side[1], out[1])


@pytest.mark.gpu
def test_stream_argument_owns_what_the_call_allocates():
    """Outputs of a call on another stream are not taken from memory that the current stream still writes."""
    w = make([1, 30], [1000, 700], 8, 2, 128, 64, 1 << 20, seed=12)
    t = [w[k].cuda() for k in ("q", "indptr", "lens", "kc", "vc", "bt")]
    want = [x.clone() for x in ola.orthros_chunk_attention(*t, 1 << 20, max_new=30)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # the current stream is behind, with writes to what it has freed
    stale = [torch.empty_like(x) for x in want for _ in range(3)]
    for x in stale:
        x.fill_(float("nan"))
    del x, stale
    got = ola.orthros_chunk_attention(*t, 1 << 20, max_new=30, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,d,new", [(8, 1, 128, 1), (8, 1, 64, 3), (32, 2, 128, 2), (6, 3, 64, 9), (16, 1, 128, 5),
                                          (16, 1, 64, 40), (5, 5, 128, 1)])
def test_long_units_of_few_heads(Hq, Hkv, d, new):
    """One sequence whose keys many CTAs share: up to one part per SM to join for a row, NaN rows among them."""
    w = make([new], [40003], Hq, Hkv, d, 64, 1 << 20, seed=18)
    want = call(w)
    check(want, plain(w, d ** -0.5))
    q = w["q"].clone()
    q[new - 1, 2] = float("nan")
    o, lse = call(dict(w, q=q))
    keep = torch.ones(new, Hq, dtype=torch.bool)
    keep[new - 1, 2] = False
    assert torch.equal(o[keep.cuda()], want[0][keep.cuda()]) and torch.equal(lse[keep.cuda()], want[1][keep.cuda()])
    assert bool(torch.isnan(o[new - 1, 2]).all()) and bool(torch.isnan(lse[new - 1, 2]))


# ---------------------------------------------------------------------------
# rows that the lanes of a warp gather (page sizes without a copy box)
# ---------------------------------------------------------------------------
def test_rows_of_all_lanes_are_ordered_before_one_lane_arrives(lib):
    """Where one lane arrives on a barrier for rows that every lane of its warp wrote and fenced, a
    warp barrier has to stand between: warp reductions and votes order no memory. Read in the
    source, since a run shows a missing order by chance at most."""
    import pathlib
    import re

    found = 0
    for path in sorted((pathlib.Path(ola.__file__).parent / "csrc").glob("*.cu")):
        text = path.read_text()
        for fence in re.finditer(r"fence_proxy_async_smem\(\);", text):
            arrive = text.find("mbar_arrive(", fence.end())
            between = text[fence.end():arrive]
            one = between.find("if (lane == 0)")
            if arrive < 0 or one < 0:
                continue  # every lane arrives for itself
            found += 1
            assert re.search(r"__sync(warp|threads)\(\);", between[:one]), \
                f"{path.name}:{text.count(chr(10), 0, fence.start()) + 1}: no warp barrier before one lane's arrival"
    assert found >= 2  # the gathered and the cleared rows of the cached attention


@pytest.mark.gpu
@pytest.mark.parametrize("page", [1, 4, 12])
def test_gathered_rows_of_long_histories(page):
    """Hundreds of gathered tiles per CTA; the same call gives the same bits every time."""
    w = make([1, 70, 1], [9001, 4000, 12345], 8, 2, 128, page, 1 << 20, seed=19)
    got = call(w, max_new=70)
    check(got, plain(w, 128 ** -0.5))
    for _ in range(5):
        again = call(w, max_new=70)
        assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.gpu
@pytest.mark.parametrize("new,total,Hq,Hkv,d,page", [
    ([1, 1, 1], [1, 5, 130], 8, 2, 128, 16),  # whole units
    ([1], [40003], 8, 1, 128, 64),            # a cut unit of few rows: a block per row joins its parts
    ([300], [5000], 32, 8, 64, 64),           # cut units of many rows
    ([40, 200], [40, 900], 4, 4, 128, 12)])   # gathered pages
def test_row_without_a_finite_logit_is_nan(new, total, Hq, Hkv, d, page):
    """A query whose logits are all -inf (an infinite channel against keys of the other sign) has no
    softmax: o is NaN, lse = log 0 = -inf, and no other row is touched."""
    w = make(new, total, Hq, Hkv, d, page, 1 << 20, seed=20)
    w["kc"][..., 7] = -w["kc"][..., 7].abs() - 0.125
    for k in w["K"]:
        k[..., 7] = -k[..., 7].abs() - 0.125
    want = call(w, max_new=max(new))
    check(want, plain(w, d ** -0.5))
    n = sum(new)
    q = w["q"].clone()
    bad = [(0, 0), (n // 2, Hq - 1), (n - 1, 1)]
    for i, h in bad:
        q[i, h, 7] = float("inf")
    o, lse = call(dict(w, q=q), max_new=max(new))
    keep = torch.ones(n, Hq, dtype=torch.bool)
    for i, h in bad:
        keep[i, h] = False
        assert bool(torch.isnan(o[i, h]).all()) and float(lse[i, h]) == -float("inf"), (i, h)
    assert torch.equal(o[keep.cuda()], want[0][keep.cuda()]) and torch.equal(lse[keep.cuda()], want[1][keep.cuda()])


# ---------------------------------------------------------------------------
# the sums and weights beside the products, to fp32
# ---------------------------------------------------------------------------
def check_fp32(got, ref, tiles, what=""):
    """The bound of the present code, in units of u = 2^-24 (an fp32 half step): a logit is off by 128 u S
    (128 products accumulated) and, with its shift, by 8 u S more (c2 = scale log2 e, m c2 and the
    difference are rounded); every exponential is ex2.approx, 4 u. A weight has one exponential for
    its key, one for each rescale of its row (the shift moves by 2^8 at least, so at most 1 + S log2(e) / 4),
    one for the join of two slots and one for each group of two parts in the merge (a part is two key
    tiles or more). The sum adds 36 values per tile, then tiles and groups: u each. lse adds logf
    (2 u |lse| with m scale taken off, which S bounds) and a sum (u). In o, P and the result are rounded
    to bf16 (2^-8 each), and P V accumulates tiles of 128 products (u each, at most 2 u where the unit truncates)."""
    u = 2.0 ** -24
    o, lse = got[0].double(), got[1].double()
    ro, rl, A, S = ref
    groups = tiles / 4 + 1
    weight = u * (136 * S + 4 * (3 + S * 1.4427 / 4 + groups) + 36 + tiles + groups)
    tol_l = weight + 4 * u * (rl.abs() + S)
    tol_o = 2.0 ** -8 * ro.abs() + (2.0 ** -8 + 2 * weight[..., None] + 256 * u * tiles) * A + 1e-30
    el, eo = ((lse - rl).abs() / tol_l).max(), ((o - ro).abs() / tol_o).max()
    assert float(el) <= 1 and float(eo) <= 1, f"{what}: lse {float(el):.3f}, o {float(eo):.3f} of the tolerance"


@pytest.mark.gpu
@pytest.mark.parametrize("qscale", [2.0 ** -6, 1.5])
@pytest.mark.parametrize("new,total,Hq,Hkv,d,page,window", CASES,
                         ids=lambda v: "-".join(map(str, v)) if isinstance(v, list) else str(v))
def test_sums_and_weights_hold_fp32(new, total, Hq, Hkv, d, page, window, qscale):
    w = make(new, total, Hq, Hkv, d, page, window, seed=sum(total) + page + 1, qscale=qscale)
    check_fp32(call(w, max_new=max(new)), plain(w, d ** -0.5), (max(total) + 127) // 128)


@pytest.mark.gpu
def test_many_parts_hold_fp32():
    """One token over 40000 keys of a single kv head: 152 parts joined."""
    for qscale in (2.0 ** -6, 1.5, 60.0):
        w = make([1], [40000], 8, 1, 128, 64, 1 << 20, seed=21, qscale=qscale)
        check_fp32(call(w), plain(w, 128 ** -0.5), 313, f"q scale {qscale}")


def test_workspace_of_a_bound_past_32_bits(lib):
    f = ola.orthros_chunk_attention_workspace_size
    assert f(2, 40, 2 ** 32 + 1, 8, 2, 128, 9, 16) == f(2, 40, 40, 8, 2, 128, 9, 16)
    assert f(2, 40, -2 ** 32 + 1, 8, 2, 128, 9, 16) == 0


@pytest.mark.gpu
def test_window_and_bound_past_32_bits():
    """A window or a bound of the new tokens beyond 32 bits is every key, every token; their lower 32
    bits mean nothing."""
    w = make([40, 1], [300, 70], 8, 2, 64, 16, 1 << 20, seed=22)
    want = call(w)
    for window, max_new in ((2 ** 32 + 1, None), (2 ** 40, None), (1 << 20, 2 ** 32 + 1), (2 ** 33 + 5, 2 ** 35)):
        got = call(dict(w, window=window), max_new=max_new)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    with pytest.raises(ola.OrthrosError):
        call(dict(w, window=-2 ** 32 + 5))
