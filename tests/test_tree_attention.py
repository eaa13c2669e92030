"""orthros_tree_attention (drafted trees over a paged cache that holds their keys) against softmax
attention in fp64. The products, sums and roundings are orthros_chunk_attention's, and so are the
tolerances (test_chunk_attention.py); a mask changes which keys a row sees, nothing of how they are added."""
import random

import numpy as np
import pytest
import torch

import efficient_long_context_gb300 as ola
from tests.test_chunk_attention import check, make

P = 1 << 12


@pytest.fixture(scope="module")
def lib():
    from efficient_long_context_gb300 import build

    build.build()
    return ola.load_library()


def _call(lib, **o):
    a = dict(q=P, qi=P, kl=P, tm=P, mw=1, kc=P, vc=P, bt=P, B=2, n=3, mn=2, Hq=4, Hkv=2, d=64, w=8, sc=0.1, dt=0, mp=4, ps=16,
             np_=8, o=P, lse=P, ws=P, wsb=1 << 30)
    a.update(o)
    return lib.orthros_tree_attention(a["q"], a["qi"], a["kl"], a["tm"], a["mw"], a["kc"], a["vc"], a["bt"], a["B"], a["n"],
                                      a["mn"], a["Hq"], a["Hkv"], a["d"], a["w"], a["sc"], a["dt"], a["mp"], a["ps"], a["np_"],
                                      a["o"], a["lse"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("over,code", [
    (dict(mw=0), 1), (dict(mw=9), 1), (dict(tm=None), 1), (dict(tm=P + 2), 1), (dict(B=-1), 1), (dict(n=-1), 1), (dict(B=0), 1),
    (dict(mn=0), 1), (dict(Hq=3), 1), (dict(d=96), 2), (dict(dt=1), 2), (dict(Hq=258, Hkv=2), 2), (dict(w=0), 1),
    (dict(sc=0.0), 1), (dict(sc=float("nan")), 1), (dict(mp=0), 1), (dict(ps=0), 1), (dict(np_=0), 1), (dict(np_=1 << 28), 2),
    (dict(ws=None), 4), (dict(wsb=1024), 4), (dict(ws=P + 16), 1), (dict(q=None), 1), (dict(o=None), 1), (dict(kc=None), 1),
    (dict(qi=None), 1), (dict(kl=None), 1), (dict(bt=None), 1), (dict(q=P + 8), 1)])
def test_refusals(lib, over, code):
    assert _call(lib, **over) == code
    assert ola.orthros_last_error() != ""


def test_workspace_size(lib):
    f = ola.orthros_tree_attention_workspace_size
    assert 0 < f(32, 32, 1, 32, 8, 128, 512, 64) < f(32, 1000, 60, 32, 8, 128, 512, 64)
    assert f(1, 1000, 1 << 40, 4, 2, 64, 16, 64) == f(1, 1000, 256, 4, 2, 64, 16, 64)  # a tree has no more
    assert f(1, 4, 0, 4, 2, 64, 1, 64) == 0 and f(1, 4, 4, 4, 2, 32, 1, 64) == 0


# ---------------------------------------------------------------------------
# the CTAs' shares of weighed key tiles, replayed on the CPU with the kernel's constants
# ---------------------------------------------------------------------------
def share_out(units, heads, per_lane, single, pair, min_tiles, snap_tiles):
    """units: (key tiles, two row tiles?) of one kv head. Checks that the shares of a lane of `heads` kv
    heads cover every tile once and in whole tiles, that none is empty, and that a unit's parts are those its
    first CTA counts; returns the largest share's cost beside an equal one's."""
    cost = [pair if two else single for _, two in units]
    start = np.concatenate([[0], np.cumsum([n * w for (n, _), w in zip(units, cost)])]).tolist()
    tiles = start[-1]
    total = heads * tiles
    eff = max(1, min(per_lane, total // (min_tiles * single)))
    snap = 0
    while snap < snap_tiles * single and 4 * (snap + 1) * eff <= total:
        snap += 1

    def moved(x, u0, n, w):
        return u0 if x - u0 <= snap else u0 + n if u0 + n - x <= snap else u0 + (x - u0) // w * w

    def unit_of(x):
        h = x // tiles
        return h, max(i for i in range(len(units)) if units[i][0] > 0 and start[i] <= x - h * tiles)

    def end(x):
        if x >= total:
            return total
        h, u = unit_of(x)
        return moved(x, h * tiles + start[u], units[u][0] * cost[u], cost[u])

    borders = [end(total * j // eff) for j in range(eff + 1)]
    seen, parts, counted = set(), {}, {}
    for j in range(eff):
        x, x1 = borders[j], borders[j + 1]
        assert x < x1, "an empty share"
        cut = 0
        while x < x1:
            h, u = unit_of(x)
            u0, n, w = h * tiles + start[u], units[u][0], cost[u]
            a = (x - u0) // w
            assert (x - u0) % w == 0
            m = min(n - a, min(x1 - x, n * w) // w)
            assert m > 0
            new = {(h, u, t) for t in range(a, a + m)}
            assert not new & seen
            seen |= new
            if a > 0 or a + m < n:
                cut += 1
                parts.setdefault((h, u), []).append(j)
                if a == 0:
                    inside = [k for k in range(j + 1, eff) if moved(total * k // eff, u0, n * w, w) < u0 + n * w]
                    counted[(h, u)] = list(range(j, j + 1)) + [k for i, k in enumerate(inside) if k == j + 1 + i]
            x += m * w
        assert cut <= 2
    assert len(seen) == heads * sum(n for n, _ in units)
    assert parts == counted
    return max(b - a for a, b in zip(borders, borders[1:])), total / eff


def test_shares_of_weighed_tiles():
    import pathlib
    import re

    text = (pathlib.Path(ola.__file__).parent / "csrc" / "chunk_attn.cu").read_text()
    single, pair, min_tiles, snap = (int(re.search(rf"{k} = (\d+)", text).group(1)) for k in
                                     ("kSingleCost", "kPairCost", "kMinTiles", "kSnap"))
    r = random.Random(1)
    for _ in range(400):
        units = [(r.choice([0, 1, 2, r.randint(1, 5), r.randint(1, 60)]), r.random() < 0.5) for _ in range(r.randint(1, 32))]
        if any(n for n, _ in units):
            most, even = share_out(units, r.choice([1, 1, 2, 3, 7]), r.choice([1, 2, 3, 9, 19, 38, 76, 152]), single, pair,
                                   min_tiles, snap)
            assert most <= 1.5 * even + pair + 1


# ---------------------------------------------------------------------------
# GPU parity
# ---------------------------------------------------------------------------
def tree_masks(new, seed, kind="tree"):
    """Rows of truth values [nb, nb] per sequence."""
    r = random.Random(seed)
    out = []
    for nb in new:
        m = torch.zeros(nb, nb, dtype=torch.bool)
        if kind == "any":  # any mask: later tokens, rows without themselves, empty rows
            m = torch.tensor([[r.random() < 0.3 for _ in range(nb)] for _ in range(nb)], dtype=torch.bool).view(nb, nb)
            if nb > 2:
                m[1] = False
        else:
            for i in range(nb):
                p = r.randint(-1, i - 1) if kind == "tree" else i - 1  # else: a chain
                if p >= 0:
                    m[i] = m[p]
                m[i, i] = True
        out.append(m)
    return out


def words_of(masks, words, junk=False):
    rows = []
    for m in masks:
        for row in m.tolist():
            x = sum(1 << j for j, s in enumerate(row) if s)
            if junk:  # bits of tokens that the tree does not have
                x |= ((1 << 32 * words) - 1) & ~((1 << len(row)) - 1)
            rows.append([(x >> 32 * w) & 0xFFFFFFFF for w in range(words)])
    a = np.array(rows, dtype=np.uint32).reshape(-1, words)
    return torch.from_numpy(a.view(np.int32))


def seen_keys(m, L, window):
    """[nb, L + nb] truth values: what the rows of a tree see."""
    nb = m.shape[0]
    t = L + m.sum(-1).clamp(min=1) - 1
    j = torch.arange(L)
    ctx = j[None, :] > t[:, None] - window
    return torch.cat([ctx, m & (t[None, :] > t[:, None] - window)], 1)


def plain(w, masks, scale):
    """fp64 (o, lse, A, S) as test_chunk_attention.plain; a row without a key has o = 0, lse = -inf."""
    q = w["q"].cuda().double()
    n, Hq, d = q.shape
    o, lse, A, S = (torch.zeros(n, Hq, d, dtype=torch.float64, device="cuda"), torch.zeros(n, Hq, dtype=torch.float64, device="cuda"),
                    torch.zeros(n, Hq, d, dtype=torch.float64, device="cuda"), torch.zeros(n, Hq, dtype=torch.float64, device="cuda"))
    i0 = 0
    for b, (nb, T) in enumerate(zip(w["new"], w["total"])):
        if nb == 0:
            continue
        K, V = w["K"][b].cuda().double(), w["V"][b].cuda().double()
        g = Hq // K.shape[1]
        seen = seen_keys(masks[b], T - nb, w["window"]).cuda()
        for h in range(Hq):
            qq, kk, vv = q[i0:i0 + nb, h], K[:, h // g], V[:, h // g]
            z = (qq @ kk.T * scale).masked_fill(~seen, float("-inf"))
            lse[i0:i0 + nb, h] = torch.logsumexp(z, -1)
            p = torch.softmax(z, -1).nan_to_num(0.0)
            o[i0:i0 + nb, h], A[i0:i0 + nb, h] = p @ vv, p @ vv.abs()
            S[i0:i0 + nb, h] = (qq.abs() @ kk.abs().T * scale).masked_fill(~seen, 0).amax(-1)
        i0 += nb
    return o, lse, A, S


def call(w, mask, **kw):
    return ola.orthros_tree_attention(w["q"].cuda(), w["indptr"].cuda(), w["lens"].cuda(), mask.cuda(), w["kc"].cuda(),
                                      w["vc"].cuda(), w["bt"].cuda(), w["window"], None, **kw)


def check_tree(got, ref, what=""):
    empty = torch.isneginf(ref[1])
    if bool(empty.any()):
        assert not bool(got[0][empty].any()) and bool(torch.isneginf(got[1][empty]).all()), what + ": rows without a key"
    rows = ~empty
    if bool(rows.any()):
        check([t[rows] for t in got], [t[rows] for t in ref], what)


BIG = 1 << 20
CASES = [
    # new, total, Hq, Hkv, d, page, window
    ([1], [1], 1, 1, 64, 64, BIG),
    ([2], [2], 32, 8, 128, 64, BIG),
    ([25], [25], 4, 2, 128, 16, BIG),
    ([25], [3000], 32, 8, 128, 64, BIG),
    ([64], [5000], 32, 8, 128, 64, BIG),
    ([33], [160], 8, 2, 64, 8, 1),
    ([33], [161], 8, 2, 64, 8, 2),
    ([60], [700], 32, 8, 128, 16, 7),
    ([60, 0, 1, 17], [700, 9, 128, 17], 32, 8, 128, 16, 100),
    ([9, 31, 32, 33, 63, 64, 65], [130, 127, 128, 129, 500, 64, 1000], 8, 2, 128, 24, BIG),
    ([128], [400], 1, 1, 64, 32, 33),
    ([256], [1000], 4, 2, 128, 64, BIG),
    ([256, 3, 200], [300, 2000, 200], 32, 8, 64, 64, 90),
    ([256], [511], 16, 1, 128, 64, BIG),  # several units of one sequence
    ([40, 9], [45, 260], 12, 1, 64, 16, BIG),
    ([3, 2], [130, 5], 128, 1, 64, 8, BIG),
    ([7, 29], [300, 700], 24, 12, 64, 16, 200),
    ([40, 1, 30], [900, 2000, 300], 10, 5, 128, 64, BIG),
    ([20, 11], [300, 7 + 11], 8, 2, 128, 1, BIG),  # page sizes without a copy box
    ([60], [300], 4, 4, 64, 12, 13),
]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["tree", "any"])
@pytest.mark.parametrize("new,total,Hq,Hkv,d,page,window", CASES,
                         ids=lambda v: "-".join(map(str, v)) if isinstance(v, list) else str(v))
def test_parity(new, total, Hq, Hkv, d, page, window, kind):
    w = make(new, total, Hq, Hkv, d, page, window, seed=sum(total) + page)
    masks = tree_masks(new, seed=sum(new), kind=kind)
    words = (max(new) + 31) // 32
    mask = words_of(masks, words, junk=True)
    ws = torch.empty(ola.orthros_tree_attention_workspace_size(len(new), sum(new), max(new), Hq, Hkv, d, w["bt"].shape[1], page),
                     dtype=torch.uint8, device="cuda")
    got = call(w, mask, max_new=max(new), workspace=ws)
    assert ola.orthros_check(ws) == (0, 0)
    check_tree(got, plain(w, masks, d ** -0.5))
    # the same bits again, with more mask words than the trees need, and another bound of the tokens
    again = call(w, words_of(masks, min(words + 1, 8)))
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.gpu
@pytest.mark.parametrize("new,total,Hq,Hkv,d,page,window", [c for c in CASES if c[6] >= max(c[0])],
                         ids=lambda v: "-".join(map(str, v)) if isinstance(v, list) else str(v))
def test_a_chain_is_the_chunk_attention(new, total, Hq, Hkv, d, page, window):
    """Tokens that hang one below the other see what consecutive ones see."""
    w = make(new, total, Hq, Hkv, d, page, window, seed=sum(total))
    masks = tree_masks(new, 0, kind="chain")
    got = call(w, words_of(masks, (max(new) + 31) // 32))
    want = ola.orthros_chunk_attention(w["q"].cuda(), w["indptr"].cuda(), w["lens"].cuda(), w["kc"].cuda(), w["vc"].cuda(),
                                       w["bt"].cuda(), window)
    ref = plain(w, masks, d ** -0.5)
    check(got, ref)
    check(want, ref)


@pytest.mark.gpu
@pytest.mark.parametrize("B", [40, 300])
def test_many_sequences(B):
    """More sequences than a CTA lists itself: the plan kernel."""
    r = random.Random(B)
    new = [r.choice([0, 1, 5, 40, 64]) for _ in range(B)]
    total = [n + r.randint(0, 400) for n in new]
    w = make(new, total, 16, 4, 64, 16, 150, seed=B)
    masks = tree_masks(new, seed=B)
    check_tree(call(w, words_of(masks, 2)), plain(w, masks, 64 ** -0.5))


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(12))
def test_mixed_batches(seed):
    """Units of one and of two row tiles side by side, whose key tiles count differently in the CTAs' shares:
    many borders in many places, every one a whole tile."""
    r = random.Random(seed)
    B, g, Hkv = r.randint(2, 32), r.choice([1, 4, 8, 16]), r.choice([1, 2, 3, 8])
    tt = 128 // g
    new = [r.choice([1, tt, min(tt + 1, 256), r.randint(1, min(2 * tt, 256)), r.randint(0, 256)]) for _ in range(B)]
    total = [n + r.choice([0, r.randint(0, 200), r.randint(0, 3000)]) for n in new]
    window = r.choice([1 << 20, r.randint(1, 2000)])
    w = make(new, total, g * Hkv, Hkv, 64, r.choice([8, 16, 64]), window, seed=seed)
    masks = tree_masks(new, seed=seed, kind=r.choice(["tree", "any"]))
    check_tree(call(w, words_of(masks, 8)), plain(w, masks, 0.125), f"{new} {total}")


@pytest.mark.gpu
@pytest.mark.parametrize("new,total,Hq,Hkv", [([9], [9], 4, 1), ([70], [5000], 8, 1), ([70] * 40, [80] * 40, 4, 2)])
def test_rows_without_a_key(new, total, Hq, Hkv):
    """No bit and no cached key in the window: zeros and -inf. A window of 1 leaves an empty row the key
    at its own position alone: none of the cached ones."""
    for window, hist in ((1, None), (1 << 20, 0)):
        tot = total if hist is None else list(new)
        w = make(new, tot, Hq, Hkv, 64, 16, window, seed=5)
        masks = tree_masks(new, 3)
        for m in masks:
            m[2] = False
        got = call(w, words_of(masks, (max(new) + 31) // 32))
        ref = plain(w, masks, 0.125)
        rows = np.concatenate([[0], np.cumsum(new)])[:-1] + 2
        assert bool(torch.isneginf(ref[1][rows]).all())
        check_tree(got, ref, f"window {window}")


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,new,total", [(4, 4, [5], [4000]), (32, 8, [40], [600]), (8, 1, [33], [33])])
def test_row_without_a_finite_logit_is_nan(Hq, Hkv, new, total):
    """A row that sees keys, but whose logits are all -inf, has no softmax (o NaN, lse -inf), unlike one
    that sees none."""
    w = make(new, total, Hq, Hkv, 64, 16, 1 << 20, seed=1)
    for t in (*w["K"], w["kc"]):
        t.copy_(torch.where(torch.isnan(t), t, t.float().abs().clamp(min=0.5).to(t.dtype)))
    q = w["q"].clone()
    q[3, 1] = float("-inf")
    masks = tree_masks(new, 2)
    got = call(dict(w, q=q), words_of(masks, 2))
    keep = torch.ones(sum(new), Hq, dtype=torch.bool, device="cuda")
    keep[3, 1] = False
    ref = plain(w, masks, 0.125)
    check([t[keep] for t in got], [t[keep] for t in ref])
    assert bool(torch.isnan(got[0][3, 1]).all()) and float(got[1][3, 1]) == float("-inf")


@pytest.mark.gpu
def test_rows_behind_the_last_sequence_stay():
    new, total = [9, 20], [300, 150]
    for more in (1, 500):
        w = make(new, total, 8, 2, 128, 16, 1 << 20, seed=7)
        masks = tree_masks(new, 7)
        q = torch.cat([w["q"], torch.full((more, 8, 128), float("nan"), dtype=torch.bfloat16)])
        mask = torch.cat([words_of(masks, 2), torch.full((more, 2), -1, dtype=torch.int32)])
        o = torch.full((29 + more, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((29 + more, 8), 7.0, device="cuda")
        call(dict(w, q=q), mask, max_new=20, out=(o, lse))
        check((o[:29], lse[:29]), plain(w, masks, 128 ** -0.5))
        assert bool((o[29:] == 7).all()) and bool((lse[29:] == 7).all())


@pytest.mark.gpu
@pytest.mark.parametrize("B", [3, 40])
def test_bad_lengths_and_pages(B):
    new, total = [9, 20, 5] + [1] * (B - 3), [300, 150, 70] + [10] * (B - 3)
    w = make(new, total, 8, 2, 64, 16, 1 << 20, seed=8)
    masks = tree_masks(new, 8)
    mask, ref = words_of(masks, 1), plain(w, masks, 0.125)
    ws = torch.empty(ola.orthros_tree_attention_workspace_size(B, sum(new), 20, 8, 2, 64, w["bt"].shape[1], 16), dtype=torch.uint8,
                     device="cuda")

    def run(bits, nan_rows, **over):
        got = call(dict(w, **over), mask, max_new=over.pop("max_new", 20), workspace=ws)
        assert ola.orthros_check(ws)[1] == bits
        nan = torch.zeros(sum(new), dtype=torch.bool, device="cuda")
        nan[nan_rows] = True
        assert bool(torch.isnan(got[0][nan]).all()) and bool(torch.isnan(got[1][nan]).all())
        check([t[~nan] for t in got], [t[~nan] for t in ref]) if not bool(nan.all()) else None

    all_rows = list(range(sum(new)))
    lens = lambda b, v: torch.tensor(total[:b] + [v] + total[b + 1:], dtype=torch.int32)
    run(0, [])
    run(4, list(range(9, 29)), lens=lens(1, 19))        # fewer cached tokens than new ones
    run(4, list(range(9, 29)), lens=lens(1, 1 << 20))   # past the block table
    run(4, list(range(9, 29)), lens=lens(1, -1))
    bad = w["indptr"].clone()
    bad[1] = 40
    run(4, all_rows, indptr=bad)
    bad = w["indptr"].clone()
    bad[B] = sum(new) + 1
    run(4, all_rows, indptr=bad)
    run(4, all_rows, indptr=torch.full_like(bad, -1))   # a refused plan
    # a page of cached keys that does not exist: all rows of the sequence; one of the tree: rows that see its tokens
    for pid in (-1, 10 ** 6):
        bt = w["bt"].clone()
        bt[0, 3] = pid
        run(2, list(range(9)), bt=bt)
    bt = w["bt"].clone()
    bt[1, 9] = -1  # keys 144 .. 149: tokens 14 .. 19 of the second tree
    sees = masks[1][:, 14:].any(1)
    run(2, [9 + i for i in range(20) if sees[i]], bt=bt)
    # a tree larger than the bound
    got = call(w, mask, max_new=9, workspace=ws)
    assert ola.orthros_check(ws)[1] == 4 and bool(torch.isnan(got[0][9:29]).all())


@pytest.mark.gpu
def test_graph_replays_growing_lengths_and_a_side_stream():
    new = [12, 5]
    w = make(new, [600, 300], 8, 2, 128, 16, 1 << 20, seed=9)
    masks = tree_masks(new, 9)
    dev = {k: w[k].cuda() for k in ("q", "indptr", "lens", "kc", "vc", "bt")}
    mask = words_of(masks, 1).cuda()
    ws = torch.empty(ola.orthros_tree_attention_workspace_size(2, 17, 12, 8, 2, 128, w["bt"].shape[1], 16), dtype=torch.uint8,
                     device="cuda")

    def attend(**kw):
        return ola.orthros_tree_attention(dev["q"], dev["indptr"], dev["lens"], mask, dev["kc"], dev["vc"], dev["bt"], 1 << 20,
                                          max_new=12, **kw)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = attend(workspace=ws)
    for lens in ([600, 300], [13, 5], [590, 299]):
        dev["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        assert ola.orthros_check(ws) == (0, 0)
        v = dict(w, total=lens, K=[k[:n] for k, n in zip(w["K"], lens)], V=[x[:n] for x, n in zip(w["V"], lens)])
        check(got, plain(v, masks, 128 ** -0.5))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = attend(stream=side)
    side.synchronize()
    assert torch.equal(other[0], got[0]) and torch.equal(other[1], got[1])


@pytest.mark.gpu
def test_empty_calls():
    z = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt, device="cuda")
    kc = z(2, 16, 2, 64, dt=torch.bfloat16)
    o, lse = ola.orthros_tree_attention(z(0, 4, 64, dt=torch.bfloat16), z(3), z(2), z(0, 1), kc, kc, z(2, 1), 8)
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)
    # rows, but no sequence has any
    out = (torch.ones(3, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(3, 4, device="cuda"))
    ws = torch.empty(ola.orthros_tree_attention_workspace_size(2, 3, 3, 4, 2, 64, 1, 16), dtype=torch.uint8, device="cuda")
    ola.orthros_tree_attention(z(3, 4, 64, dt=torch.bfloat16), z(3), z(2), z(3, 1), kc, kc, z(2, 1), 8, out=out, workspace=ws)
    assert ola.orthros_check(ws) == (0, 0) and bool((out[0] == 1).all()) and bool((out[1] == 1).all())


@pytest.mark.gpu
def test_long_cache():
    """Offsets past 32 bits: pages in the upper half of a pool of more than 2^32 elements."""
    page, Hkv, d = 64, 8, 128
    pages = (5 << 30) // (page * Hkv * d)  # 10 GB a cache
    kc = torch.empty((pages, page, Hkv, d), dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    w = make([30], [500], 16, Hkv, d, page, 1 << 20, seed=10)
    used = [int(x) for x in w["bt"][0]]
    far = [pages - 1 - 3 * i for i in range(len(used))]
    for u, f in zip(used, far):
        kc[f], vc[f] = w["kc"][u].cuda(), w["vc"][u].cuda()
    masks = tree_masks([30], 10)
    bt = torch.tensor([far], dtype=torch.int32, device="cuda")
    got = ola.orthros_tree_attention(w["q"].cuda(), w["indptr"].cuda(), w["lens"].cuda(), words_of(masks, 1).cuda(), kc, vc, bt,
                                     1 << 20)
    check(got, plain(w, masks, d ** -0.5))
    # the commit's rows lie there too
    want = kc.flatten(0, 1)[far[7] * page + (470 + 5) % page].clone()
    lens = ola.orthros_tree_commit(kc, vc, bt, w["indptr"].cuda(), w["lens"].cuda(),
                                   torch.tensor([[5]], dtype=torch.int32, device="cuda"),
                                   torch.tensor([1], dtype=torch.int32, device="cuda"))
    assert lens.tolist() == [471] and torch.equal(kc.flatten(0, 1)[far[7] * page + 470 % page], want)


@pytest.mark.gpu
@pytest.mark.parametrize("page", [8, 16, 64, 128, 12])  # the last one without a copy box
@pytest.mark.parametrize("B", [2, 40])  # without and with a plan kernel
def test_every_page_id_outside_the_pool_is_reported(B, page):
    new, total = [9, 20] + [1] * (B - 2), [300, 150] + [10] * (B - 2)
    w = make(new, total, 8, 2, 128, page, 1 << 20, seed=20)
    masks = tree_masks(new, 20)
    mask, ref, pool = words_of(masks, 1), plain(w, masks, 128 ** -0.5), w["kc"].shape[0]
    ws = torch.empty(ola.orthros_tree_attention_workspace_size(B, sum(new), 20, 8, 2, 128, w["bt"].shape[1], page), dtype=torch.uint8,
                     device="cuda")
    for pid in (-2 ** 31, -2 ** 31 + 1, -2, -1, pool, 2 ** 31 - 1):
        bt = w["bt"].clone()
        bt[0, 140 // page] = pid
        o, lse = call(dict(w, bt=bt), mask, max_new=20, workspace=ws)
        assert ola.orthros_check(ws) == (5, 2), pid
        assert bool(torch.isnan(o[:9]).all()) and bool(torch.isnan(lse[:9]).all()), pid
        check_tree((o[9:], lse[9:]), [r[9:] for r in ref], f"page id {pid}")
