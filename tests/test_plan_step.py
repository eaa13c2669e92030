"""orthros_plan_step and orthros_tree_commit against plain Python: whole numbers and moved rows, so every
comparison is for equality."""
import random

import pytest
import torch

import efficient_long_context_gb300 as ola

P = 1 << 12
LENGTH, PAGE, POSITION, NO_PAGES = 4, 2, 1, 32


@pytest.fixture(scope="module")
def lib():
    from efficient_long_context_gb300 import build

    build.build()
    return ola.load_library()


def _plan(lib, **o):
    a = dict(cl=P, nl=P, ph=P, fc=P, pa=P, mt=8, fp=P, bt=P, B=2, n=3, mp=4, ps=16, np_=8, qi=P, kl=2 * P, lo=P, pho=P, fco=P, ts=P, tp=P,
             sl=P, tm=P, ws=P, wsb=256)
    a.update(o)
    return lib.orthros_plan_step(a["cl"], a["nl"], a["ph"], a["fc"], a["pa"], a["mt"], a["fp"], a["bt"], a["B"], a["n"], a["mp"],
                                 a["ps"], a["np_"], a["qi"], a["kl"], a["lo"], a["pho"], a["fco"], a["ts"], a["tp"], a["sl"], a["tm"],
                                 a["ws"], a["wsb"], None)


@pytest.mark.parametrize("over,code", [
    (dict(B=0), 1), (dict(B=8193), 2), (dict(n=-1), 1), (dict(mp=0), 1), (dict(ps=0), 1), (dict(np_=0), 1),
    (dict(np_=1 << 28), 2), (dict(mp=1 << 28), 2), (dict(mt=-1), 1), (dict(mt=257), 1), (dict(pa=None), 1), (dict(tm=None), 1),
    (dict(ws=None), 4), (dict(wsb=8), 4), (dict(ws=P + 8), 1), (dict(cl=None), 1), (dict(nl=None), 1), (dict(ph=None), 1),
    (dict(fc=None), 1), (dict(fp=None), 1), (dict(bt=None), 1), (dict(qi=None), 1), (dict(kl=None), 1), (dict(pho=None), 1),
    (dict(fco=None), 1), (dict(ts=None), 1), (dict(tp=None), 1), (dict(sl=None), 1), (dict(cl=P + 2), 1),
    (dict(kl=P), 1), (dict(kl=P, lo=None), 1), (dict(lo=2 * P), 1), (dict(lo=P + 2), 1)])
def test_plan_refusals(lib, over, code):
    assert _plan(lib, **over) == code
    assert ola.orthros_last_error() != ""


def _commit(lib, **o):
    a = dict(kc=P, vc=P, la=1, bt=P, qi=P, kl=2 * P, ac=P, na=P, mo=4, B=2, Hkv=2, d=64, dt=0, mp=4, ps=16, np_=8, cl=P + 64,
             ws=P, wsb=256)
    a.update(o)
    return lib.orthros_tree_commit(a["kc"], a["vc"], a["la"], a["bt"], a["qi"], a["kl"], a["ac"], a["na"], a["mo"], a["B"],
                                   a["Hkv"], a["d"], a["dt"], a["mp"], a["ps"], a["np_"], a["cl"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("over,code", [
    (dict(la=0), 1), (dict(la=65536), 1), (dict(mo=0), 1), (dict(mo=257), 1), (dict(B=0), 1), (dict(Hkv=0), 1), (dict(d=96), 2),
    (dict(dt=5), 1), (dict(mp=0), 1), (dict(ps=0), 1), (dict(np_=0), 1), (dict(np_=1 << 28), 2), (dict(kc=None), 1),
    (dict(vc=P + 8), 1), (dict(bt=None), 1), (dict(qi=None), 1), (dict(kl=None), 1), (dict(ac=None), 1), (dict(na=None), 1),
    (dict(cl=None), 1), (dict(cl=2 * P), 1), (dict(cl=P), 1), (dict(ws=None), 4), (dict(wsb=8), 4), (dict(ws=P + 8), 1)])
def test_commit_refusals(lib, over, code):
    assert _commit(lib, **over) == code
    assert ola.orthros_last_error() != ""


def test_binding_refusals(lib):
    z = lambda *s: torch.zeros(s, dtype=torch.int32)
    with pytest.raises(ola.OrthrosError):
        ola.orthros_plan_step(z(2), z(2), z(2), z(8), z(1), z(2, 4), 16, 3, parents=z(3))  # no max_tree
    with pytest.raises(ola.OrthrosError):
        ola.orthros_plan_step(z(2), z(2), z(2), z(8), z(1), z(2, 4), 16, 3)  # not on the GPU
    k = torch.zeros(8, 16, 2, 64)
    with pytest.raises(ola.OrthrosError):
        ola.orthros_tree_commit(k[0], k[0], z(2, 4), z(3), z(2), z(2, 4), z(2))
    with pytest.raises(ola.OrthrosError):
        ola.orthros_tree_commit(k, k, z(2, 4), z(3), z(2), z(8), z(2))


# ---------------------------------------------------------------------------
# the plan, in plain Python
# ---------------------------------------------------------------------------
def plain_plan(cl, nl, held, free, count, bt, page, n, parents, max_tree):
    """The header's rules, one sequence after the other. Lists in, a dict out; bits of the status word."""
    cl, held, free, bt = list(cl), list(held), list(free), [list(r) for r in bt]
    B, mp, pool, words = len(cl), len(bt[0]), len(free), (max_tree + 31) // 32
    bits, rows, at = 0, [], 0
    wrong = []
    for b in range(B):
        total = cl[b] + max(nl[b], 0)
        w = nl[b] < -1 or not 0 <= held[b] <= mp or \
            (nl[b] >= 0 and (cl[b] < 0 or total > mp * page or (max_tree > 0 and nl[b] > max_tree)))
        wrong.append(w)
        bits |= LENGTH if w else 0
        rows.append(at)
        at += max(nl[b], 0)
    back = sum(held[b] for b in range(B) if not wrong[b] and nl[b] == -1)
    out = dict(token_seq=[-1] * n, token_pos=[0] * n, token_slots=[-1] * n, tree_mask=[[0] * words for _ in range(n)])
    if at > n or count < 0 or count + back > pool:
        return dict(out, q_indptr=[-1] * (B + 1), kv_lens=[-1] * B, cache_lens=cl, pages_held=held, free_count=count, block_table=bt,
                    free_pages=None, bits=bits | LENGTH)
    stack = free[:count]
    for b in range(B):
        if not wrong[b] and nl[b] == -1:
            stack += bt[b][:held[b]]
    free[:len(stack)] = stack
    avail, taken = len(stack), 0
    kv, new_held = [-1] * B, list(held)
    lens = list(cl)
    short = 0  # pages that sequences without enough of them would have taken
    for b in range(B):
        if wrong[b]:
            continue
        if nl[b] == -1:
            new_held[b] = lens[b] = kv[b] = 0
            continue
        need = max(held[b], (cl[b] + nl[b] + page - 1) // page)
        lack = need - held[b]
        if lack and taken + short + lack > avail:
            short += lack
            bits |= NO_PAGES
            continue
        for i in range(held[b], need):
            bt[b][i] = stack[avail - 1 - taken]
            taken += 1
        new_held[b], kv[b] = need, cl[b] + nl[b]
        lens[b] = kv[b]
        for j in range(nl[b]):
            r = rows[b] + j
            out["token_seq"][r] = b
            place = cl[b] + j
            pg = bt[b][place // page]
            if 0 <= pg < pool:
                out["token_slots"][r] = pg * page + place % page
            else:
                bits |= PAGE
            depth, up = 0, j
            if max_tree:
                m = 0
                while True:
                    m |= 1 << up
                    to = parents[rows[b] + up]
                    if to < -1 or to >= up:
                        bits |= POSITION
                    if not 0 <= to < up:
                        break
                    up, depth = to, depth + 1
                out["tree_mask"][r] = [(m >> 32 * w) & 0xFFFFFFFF for w in range(words)]
                place = cl[b] + depth
            out["token_pos"][r] = place
    return dict(out, q_indptr=rows + [at], kv_lens=kv, cache_lens=lens, pages_held=new_held, free_count=avail - taken, block_table=bt,
                free_pages=free, bits=bits)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def run(case, in_place=False, **kw):
    """The call on a case's lists; its outputs as lists like plain_plan's."""
    cl, nl, held, free, count, bt, page, n, parents, max_tree = case
    t = [i32(cl), i32(nl), i32(held), i32(free), i32([count]), i32(bt)]
    out = None
    if in_place:
        b = ola.orthros_plan_step_buffers(len(cl), n, max_tree)
        out = b._replace(cache_lens=t[0], pages_held=t[2], free_count=t[4])
    ws = torch.full((256,), 255, dtype=torch.uint8, device="cuda")
    plan = ola.orthros_plan_step(*t, page, n, parents=i32(parents) if max_tree else None, max_tree=max_tree, out=out, workspace=ws,
                                 **kw)
    got = {k: getattr(plan, k).tolist() for k in plan._fields if getattr(plan, k) is not None}
    got["free_count"] = got["free_count"][0]
    got["tree_mask"] = [[x % 2 ** 32 for x in r] for r in got["tree_mask"]] if max_tree else [[] for _ in range(n)]
    return dict(got, block_table=t[5].tolist(), free_pages=t[3].tolist(), bits=ola.orthros_check(ws)[1])


def check(case, **kw):
    want, got = plain_plan(*case), run(case, **kw)
    for k, v in want.items():
        if v is not None:  # (the stack's entries above its height are not specified once a step is refused)
            assert got[k] == v, (k, got[k], v)
    return got


def make(B, new, hist, page, seed, tree=0, ends=0.0, pad=0, extra=0):
    """Consistent state: each sequence holds the pages of its cached tokens (and `extra` more)."""
    r = random.Random(seed)
    cl = [r.randint(0, hist) for _ in range(B)]
    nl = [r.randint(0, new) for _ in range(B)]
    if tree:
        nl = [min(m, tree) for m in nl]
    held = [(c + page - 1) // page + (r.randint(0, extra) if extra else 0) for c in cl]
    mp = max((c + m + page - 1) // page for c, m in zip(cl, nl)) + 1 + extra
    nl = [-1 if r.random() < ends else m for m in nl]
    spare = sum((max(m, 0) + page - 1) // page + 1 for m in nl)
    ids = list(range(sum(held) + spare))
    r.shuffle(ids)
    bt, at = [], 0
    for h in held:
        bt.append(ids[at:at + h] + [-7] * (mp - h))
        at += h
    free = ids[at:] + [-9] * at
    n = sum(max(m, 0) for m in nl) + pad
    parents = []
    for m in nl:
        parents += [r.randint(-1, i - 1) for i in range(max(m, 0))]
    parents += [99] * pad
    return [cl, nl, held, free, spare, bt, page, n, parents, tree]


CASES = [
    # B, new, hist, page, kw
    (1, 1, 0, 1, {}), (1, 0, 100, 16, {}), (1, 5000, 300, 16, {}), (3, 7, 50, 5, dict(pad=4)), (64, 1, 3000, 64, {}),
    (1, 1, 5, 8, dict(tree=1)), (1, 256, 1000, 64, dict(tree=256)), (33, 64, 500, 16, dict(tree=64, ends=0.2, pad=100)),
    (40, 31, 500, 48, dict(tree=33, ends=0.5)), (200, 20, 100, 8, dict(ends=0.9, extra=3)), (1025, 3, 90, 16, dict(ends=0.1)),
    (2050, 9, 20, 4, dict(tree=9, pad=3000)), (8192, 1, 40, 16, dict(ends=0.01)),
]


@pytest.mark.gpu
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,new,hist,page,kw", CASES, ids=lambda v: str(v))
def test_plan(B, new, hist, page, kw, in_place):
    case = make(B, new, hist, page, seed=B + new, **kw)
    got = check(case, in_place=in_place)
    assert got["bits"] == 0


@pytest.mark.gpu
def test_plan_of_no_rows():
    case = make(5, 0, 100, 16, seed=1, ends=0.4)
    assert case[7] == 0
    check(case)


@pytest.mark.gpu
def test_plan_reports_what_cannot_be():
    base = make(6, 20, 300, 16, seed=3, tree=20)
    for k, b, v, bits in ((0, 2, -1, LENGTH), (1, 3, -2, LENGTH), (1, 3, -2 ** 31, LENGTH), (2, 1, -1, LENGTH),
                          (2, 1, 10 ** 6, LENGTH), (0, 4, 2 ** 31 - 1, LENGTH), (0, 5, 100000, LENGTH)):
        case = [list(x) if isinstance(x, list) else x for x in base]
        case[k][b] = v
        if k == 1:
            case[8] = [-1] * case[7]  # (the other sequences' rows move up)
        assert check(case)["bits"] == bits
        assert check(case, in_place=True)["bits"] == bits
    # a tree larger than the limit; its rows are padding, the other trees stay where they are
    case = make(4, 9, 100, 16, seed=4, tree=9)
    case[1][1] = max(case[1][1], 5)
    case[7] = sum(case[1]) + 2
    case[8] = [-1] * case[7]
    case[9] = 4
    assert check(case)["bits"] & LENGTH
    # more tokens than rows; a height that the stack does not have
    for change in (lambda c: c.__setitem__(7, c[7] - 1), lambda c: c.__setitem__(4, len(c[3]) + 1), lambda c: c.__setitem__(4, -1),
                   lambda c: c[1].__setitem__(0, 2 ** 31 - 1)):
        case = make(9, 7, 100, 16, seed=5)
        change(case)
        case[8] = case[8][:case[7]]
        assert check(case)["bits"] & LENGTH
        assert check(case, in_place=True)["bits"] & LENGTH
    # ended sequences that hold more pages than the pool has
    case = make(3, 2, 100, 16, seed=6)
    case[1] = [-1, -1, 1]
    case[4] = len(case[3]) - 1
    case[7], case[8] = 1, []
    assert check(case)["bits"] == LENGTH
    # parents that do not come before their tokens
    case = make(3, 6, 50, 8, seed=7, tree=6)
    case[1] = [4, 6, 3]
    case[7], case[8] = 13, [-1, 1, 7, -2] + [0] * 6 + [-1, 0, 2 ** 31 - 1]
    assert check(case)["bits"] == POSITION
    # page ids outside the pool: held ones and free ones
    case = make(3, 30, 60, 8, seed=8)
    case[5][0][0], case[3][case[4] - 1] = 10 ** 6, -5
    case[0][0], case[2][0] = max(case[0][0], 1), max(case[2][0], 1)
    assert check(case)["bits"] in (0, PAGE)


@pytest.mark.gpu
def test_plan_of_an_ended_sequence_reads_no_length():
    case = make(5, 4, 60, 8, seed=9)
    case[1][2], case[0][2] = -1, 2 ** 31 - 1
    case[1][4], case[0][4] = -1, -77
    case[7] = sum(max(m, 0) for m in case[1])
    for in_place in (False, True):
        got = check(case, in_place=in_place)
        assert got["bits"] == 0 and got["kv_lens"][2] == 0 == got["pages_held"][4]


@pytest.mark.gpu
def test_commit_after_a_refused_plan_keeps_the_lengths():
    """A refused step, and a sequence without a place in one (also one without tokens), leave cache_lens to the
    commit as they were."""
    for change, keep in ((lambda c: c.__setitem__(7, c[7] - 1), range(5)), (lambda c: c[2].__setitem__(1, -3), [1]),
                         (lambda c: c[0].__setitem__(3, 10 ** 6), [3])):
        case = make(5, 6, 40, 8, seed=10, tree=6)
        case[1] = [3, 0, 4, 0, 2]
        case[7], case[8] = 9, [-1, 0, 1, -1, 0, 0, 2, -1, -1]
        change(case)
        case[8] = case[8][:case[7]]
        got = run(case)
        lens = i32(case[0])
        kc = torch.zeros(len(case[3]), 8, 1, 64, device="cuda")
        bt = [[max(x, 0) for x in row] for row in got["block_table"]]
        ola.orthros_tree_commit(kc, kc.clone(), i32(bt), i32(got["q_indptr"]), i32(got["kv_lens"]), i32([[0]] * 5),
                                i32([1, 0, 1, 0, 1]), out=lens)
        want = [L + n if b not in keep else L for b, (L, n) in enumerate(zip(case[0], [1, 0, 1, 0, 1]))]
        assert lens.tolist() == want


@pytest.mark.gpu
@pytest.mark.parametrize("count", [0, 1, 3, 7])
def test_plan_short_of_pages(count):
    """Sequences whose pages are not all there change nothing; those that need none go on, and pages of
    ended sequences count."""
    page = 4
    cl, nl = [4, 3, 8, 0, 5, 2], [9, 1, 1, 6, 1, 1]
    held = [1, 1, 2, 0, 2, 1]
    ids = list(range(20))
    bt, at = [], 0
    for h in held:
        bt.append(ids[at:at + h] + [-1] * (6 - h))
        at += h
    case = [cl, nl, held, ids[at:at + count] + [-1] * (20 - count), count, bt, page, sum(nl), [], 0]
    got = check(case)
    assert bool(got["bits"] & NO_PAGES) == (count < 6)
    case[1] = [9, 1, 1, 6, -1, 1]
    case[7] = 18
    check(case)


@pytest.mark.gpu
def test_plan_in_a_graph_advances():
    """A captured plan with its state in place decodes: lengths grow, pages are taken as borders are
    crossed, until none is free."""
    page, B = 4, 3
    cl, held, count = i32([3, 0, 6]), i32([1, 0, 2]), i32([4])
    bt = i32([[0, -1, -1, -1], [-1] * 4, [1, 2, -1, -1]])
    free = i32([3, 4, 5, 6, -1, -1, -1])
    out = ola.orthros_plan_step_buffers(B, B)._replace(cache_lens=cl, pages_held=held, free_count=count)
    nl, ws = i32([1] * B), torch.empty(256, dtype=torch.uint8, device="cuda")
    step = lambda: ola.orthros_plan_step(cl, nl, held, free, count, bt, page, B, out=out, workspace=ws)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.synchronize()
    state = [[3, 0, 6], [1, 0, 2], [3, 4, 5, 6, -1, -1, -1], 4, bt.tolist()]
    for _ in range(7):
        graph.replay()
        want = plain_plan(state[0], [1] * B, state[1], state[2], state[3], state[4], page, B, [], 0)
        assert out.kv_lens.tolist() == want["kv_lens"] and cl.tolist() == want["cache_lens"] and held.tolist() == want["pages_held"] and count.tolist() == [want["free_count"]]
        assert out.token_slots.tolist() == want["token_slots"] and bt.tolist() == want["block_table"]
        assert ola.orthros_check(ws)[1] == want["bits"]
        state = [want["cache_lens"], want["pages_held"], want["free_pages"], want["free_count"], want["block_table"]]


# ---------------------------------------------------------------------------
# commit
# ---------------------------------------------------------------------------
def make_commit(B, layers, Hkv, d, page, dtype, nb, hist, most, seed):
    r, g = random.Random(seed), torch.Generator().manual_seed(seed)
    new = [r.randint(0, nb) for _ in range(B)]
    ctx = [r.randint(0, hist) for _ in range(B)]
    lens = [a + b for a, b in zip(new, ctx)]
    mp = max(1, max((x + page - 1) // page for x in lens))
    pool = B * mp + 2
    bt = torch.randperm(pool, generator=g)[:B * mp].view(B, mp)
    acc, cnt = [], []
    for m in new:
        k = r.randint(0, min(m, most))
        acc.append(sorted(r.sample(range(m), k)) + [-5] * (most - k))
        cnt.append(k)
    kc, vc = (torch.randn(layers, pool, page, Hkv, d, generator=g).to(dtype) for _ in range(2))
    indptr = [0]
    for m in new:
        indptr.append(indptr[-1] + m)
    return dict(kc=kc, vc=vc, bt=bt, indptr=indptr, lens=lens, acc=acc, cnt=cnt, ctx=ctx, page=page)


def plain_commit(w, skip=()):
    out = []
    for c in (w["kc"], w["vc"]):
        c = c.clone()
        old = c.clone()
        for b, L in enumerate(w["ctx"]):
            for i in range(w["cnt"][b] if b not in skip else 0):
                s, t = L + w["acc"][b][i], L + i
                c[:, w["bt"][b, t // w["page"]], t % w["page"]] = old[:, w["bt"][b, s // w["page"]], s % w["page"]]
        out.append(c)
    return out


def call_commit(w, ws=None, **kw):
    k, v = w["kc"].cuda(), w["vc"].cuda()
    lens = ola.orthros_tree_commit(k, v, w["bt"].to(torch.int32).cuda(), i32(w["indptr"]), i32(w["lens"]), i32(w["acc"]),
                                   i32(w["cnt"]), workspace=ws, **kw)
    return k.cpu(), v.cpu(), lens.tolist()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("B,layers,Hkv,d,page,nb,hist,most", [
    (1, 1, 1, 64, 1, 1, 0, 1), (1, 1, 8, 128, 16, 40, 100, 40), (5, 3, 2, 64, 5, 30, 77, 9), (33, 2, 3, 128, 64, 64, 200, 17),
    (3, 1, 16, 128, 8, 256, 30, 256), (40, 1, 1, 64, 16, 6, 50, 3), (300, 1, 1, 64, 4, 8, 9, 8)])
def test_commit(B, layers, Hkv, d, page, nb, hist, most, dtype):
    w = make_commit(B, layers, Hkv, d, page, dtype, nb, hist, most, seed=B + nb)
    ws = torch.full((256,), 255, dtype=torch.uint8, device="cuda")
    k, v, lens = call_commit(w, ws)
    assert ola.orthros_check(ws) == (0, 0)
    want = plain_commit(w)
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])
    assert lens == [a + b for a, b in zip(w["ctx"], w["cnt"])]


@pytest.mark.gpu
def test_commit_reports_bad_paths():
    base = make_commit(6, 2, 2, 64, 8, torch.float32, 20, 60, 8, seed=11)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    b = max(range(6), key=lambda s: base["cnt"][s])
    assert base["cnt"][b] >= 3
    nb = base["indptr"][b + 1] - base["indptr"][b]

    def bad(bits, **change):
        w = dict(base, acc=[list(r) for r in base["acc"]], cnt=list(base["cnt"]), lens=list(base["lens"]), bt=base["bt"].clone())
        for name, (at, v) in change.items():
            if name == "acc":
                w["acc"][b][at] = v
            elif name == "bt":
                w["bt"][b, at] = v
            else:
                w[name][b] = v
        k, v, lens = call_commit(w, ws, out=i32([77] * 6))
        assert ola.orthros_check(ws)[1] == bits, change
        ok = dict(w, bt=base["bt"])
        want = plain_commit(ok, skip=(b,))
        assert torch.equal(k, want[0]) and torch.equal(v, want[1])
        want = [L + (n if s != b else 0) for s, (L, n) in enumerate(zip(base["ctx"], base["cnt"]))]
        if "lens" in change:
            want[b] = 77  # left as it was
        assert lens == want

    bad(POSITION, acc=(1, base["acc"][b][0]))  # does not ascend
    bad(POSITION, acc=(0, -1))
    bad(POSITION, acc=(base["cnt"][b] - 1, nb))
    bad(POSITION, acc=(2, 2 ** 31 - 1))
    bad(LENGTH, cnt=(0, -1))
    bad(LENGTH, cnt=(0, 9))
    bad(LENGTH, lens=(0, nb - 1))
    bad(LENGTH, lens=(0, 10 ** 6))
    pg = (base["ctx"][b] + base["acc"][b][1]) // 8
    bad(PAGE, bt=(pg, -1))
    bad(PAGE, bt=(pg, 10 ** 6))


@pytest.mark.gpu
def test_commit_in_a_graph_and_on_a_stream():
    w = make_commit(7, 2, 2, 128, 16, torch.bfloat16, 12, 40, 6, seed=12)
    want = plain_commit(w)
    k, v = w["kc"].cuda(), w["vc"].cuda()
    args = [w["bt"].to(torch.int32).cuda(), i32(w["indptr"]), i32(w["lens"]), i32(w["acc"]), i32(w["cnt"])]
    out, ws = torch.zeros(7, dtype=torch.int32, device="cuda"), torch.empty(256, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ola.orthros_tree_commit(k, v, *args, out=out, workspace=ws)
    assert torch.equal(k.cpu(), w["kc"])
    graph.replay()
    assert torch.equal(k.cpu(), want[0]) and torch.equal(v.cpu(), want[1])
    side = torch.cuda.Stream()
    k2, v2 = w["kc"].cuda(), w["vc"].cuda()
    side.wait_stream(torch.cuda.current_stream())
    lens = ola.orthros_tree_commit(k2, v2, *args, stream=side)
    side.synchronize()
    assert torch.equal(k2, k) and torch.equal(v2, v) and torch.equal(lens, out)


@pytest.mark.gpu
def test_commit_without_out_knows_no_length_of_a_sequence_without_a_place():
    """The lengths that the call allocates are -1 where the step had no place for the sequence: 0 would be the
    length of an ended one. A plan that is given them refuses those sequences and leaves their pages alone."""
    page, parents = 8, [-1, 0, 0, -1, 0, -1, 0, -1]
    bt = [[0, 1] + [-1] * 4, [2, 3] + [-1] * 4, [4] + [-1] * 5, [5, 6] + [-1] * 4]
    for third, lost in ((-1, []), (0, [1])):  # the second sequence needs a page: the third one's, if that ends
        case = [[9, 16, 5, 8], [3, 4, third, 1], [2, 2, 1, 2], [-1] * 8, 0, bt, page, 8, parents, 6]
        got = check(case)
        assert [b for b, kv in enumerate(got["kv_lens"]) if kv < 0] == lost
        kc = torch.zeros(8, 8, 1, 64, device="cuda")
        args = (kc, kc.clone(), i32([[max(x, 0) for x in row] for row in got["block_table"]]), i32(got["q_indptr"]), i32(got["kv_lens"]), i32([[0]] * 4))
        count = [1, 1, 0, 1]
        lens = ola.orthros_tree_commit(*args, i32(count)).tolist()
        want = [c + k for c, k in zip(case[0], count)]
        if not lost:
            want[2] = 0  # ended
        for b in lost:
            want[b] = -1
        assert lens == want
    # carried on: the sequence stays out of the step, its pages and table untouched
    nxt = [lens, [1, 1, 1, 1], got["pages_held"], [7] + [-1] * 7, 1, got["block_table"], 8, 4, [-1] * 4, 6]
    got = check(nxt)
    assert got["bits"] == LENGTH and got["kv_lens"][1] == -1 and got["block_table"][1] == bt[1]
    # a refused step: of every sequence
    refused = i32([-1] * 5)
    assert ola.orthros_tree_commit(*args[:3], refused, i32([-1] * 4), args[5], i32(count)).tolist() == [-1] * 4


def check_bad_page(case, b, **kw):
    """The plan of a case in which sequence b ends with a page id from outside the pool: it stays as it is, as one
    whose lengths cannot be, and the others' step is that without it."""
    as_wrong = [list(x) if isinstance(x, list) else x for x in case]
    as_wrong[1][b] = -2
    want, got = plain_plan(*as_wrong), run(case, **kw)
    want["bits"] = want["bits"] & ~LENGTH | PAGE
    for k, v in want.items():
        if v is not None:
            assert got[k] == v, (k, got[k], v)
    return got


@pytest.mark.gpu
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,new,hist,page,kw", [(3, 2, 40, 8, {}), (40, 9, 500, 16, dict(tree=9, ends=0.3, pad=7)),
                                                (9, 1, 9000, 4, dict(ends=0.5)), (1500, 4, 60, 8, dict(ends=0.2)),
                                                (600, 12, 90, 8, dict(tree=12, ends=0.1))], ids=lambda v: str(v))
def test_plan_keeps_ids_of_elsewhere_off_the_stack(B, new, hist, page, kw, in_place):
    """An ended sequence gives its pages back only if all of them are the pool's."""
    base = make(B, new, hist, page, seed=B + page, **kw)
    b = max(range(B), key=lambda s: base[2][s])
    base[1][b] = -1
    base[7] = sum(max(m, 0) for m in base[1]) + kw.get("pad", 0)
    base[8] = [-1] * base[7]
    held, pool = base[2][b], len(base[3])
    for at in sorted({0, held // 2, held - 1}):
        for pid in (-1, -2 ** 31, pool, 2 ** 31 - 1):
            case = [list(x) if isinstance(x, list) else x for x in base]
            case[5] = [list(r) for r in base[5]]
            case[5][b][at] = pid
            got = check_bad_page(case, b, in_place=in_place)
            assert got["kv_lens"][b] == -1 and got["pages_held"][b] == held and got["cache_lens"][b] == base[0][b]
            assert pid not in got["free_pages"][:got["free_count"]]
    # what it does not hold is not read
    case = [list(x) if isinstance(x, list) else x for x in base]
    case[5] = [list(r) for r in base[5]]
    case[5][b][held:] = [-2 ** 31] * (len(case[5][b]) - held)
    assert check(case, in_place=in_place)["bits"] == 0


@pytest.mark.gpu
def test_plan_reports_pages_that_it_takes_without_a_token_on_them():
    """A sequence that holds fewer pages than its cached tokens take gets the rest without new tokens of its
    own; an id from outside the pool among them is reported in that step."""
    for tree in (0, 4):
        case = [[20, 3], [0, 1], [1, 1], [5, -7, 6, 3] + [-1] * 4, 4, [[0, -1, -1, -1], [1, -1, -1, -1]], 8, 2, [-1] * 2, tree]
        want = plain_plan(*case)
        got = run(case)
        assert want["bits"] == 0 and want["block_table"][0][:3] == [0, 3, 6]  # two taken, both good
        assert got["bits"] == 0 and got["block_table"] == want["block_table"]
        for pid in (-7, 8, -2 ** 31):
            case[3][2] = pid
            want, got = plain_plan(*case), run(case)
            assert got.pop("bits") == PAGE
            want.pop("bits")
            assert all(got[k] == v for k, v in want.items() if v is not None)


def test_warps_are_converged_at_aligned_cluster_barriers(lib):
    """An aligned barrier is undefined for a warp whose lanes come apart, as behind a branch of one lane: a warp
    barrier stands directly before each. Read in the source, since a run shows its lack by chance at most."""
    import pathlib
    import re

    found = 0
    for path in sorted((pathlib.Path(ola.__file__).parent / "csrc").glob("*.cu*")):
        text = path.read_text()
        for m in re.finditer(r'asm volatile\("barrier\.cluster\.arrive[.a-z]*\.aligned', text):
            found += 1
            before = text[:m.start()].rstrip()
            assert before.endswith("__syncwarp();"), f"{path.name}:{text.count(chr(10), 0, m.start()) + 1}"
    assert found >= 1
