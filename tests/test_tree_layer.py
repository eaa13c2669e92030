"""The rotary layer with norms and drafted trees: plan, normed append, tree attention and commit as a
serving loop calls them, and the training path with norms.

Serving. A tree's token and the same token as the end of its path, decoded as consecutive tokens, read
the same bf16 queries, keys and values; each output lies within the attention contract of the exact
value (2e-2 absolute for N(0, 1) inputs), so they are 4e-2 apart at most. Cached rows are projected,
normed and rotated alike in both: two roundings to bf16 of one value, 2^-7 relative.
Gradients: the bound of test_rotary_layer.py (5e-2 of rms(ref) + |ref| + floor); the norm's gradient is
linear in the rotation's, with a factor r w of about 1 here.
"""
import random

import numpy as np
import pytest
import torch

import efficient_long_context_gb300 as ola
from efficient_long_context_gb300.rotary_layer import RotaryLayer

D_MODEL = 256


def make_layer(Hq, Hkv, d, window, layout, seed, normed, rot=None, device="cuda"):
    g = torch.Generator().manual_seed(seed)
    w = (torch.randn((Hq + 2 * Hkv) * d, D_MODEL, generator=g) / D_MODEL ** 0.5).bfloat16().to(device)
    aff = []
    for _ in range(2):
        aff += [(1 + 0.1 * torch.randn(Hq, d, generator=g)).to(device), (0.1 * torch.randn(Hq, d, generator=g)).to(device)]
    freq, amp = ola.orthros_rotary_frequencies(rot or d, 10000.0)
    norms = [(1 + 0.2 * torch.randn(d, generator=g)).to(device) for _ in range(2)] if normed else [None, None]
    return RotaryLayer(w, aff, freq, Hq, Hkv, d, window, layout, amp, *norms), g


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Server:
    """Lengths, pages and caches of a batch, all on the GPU."""

    def __init__(self, layer, B, page, pages):
        self.layer, self.B, self.page = layer, B, page
        self.kc = torch.full((pages, page, layer.Hkv, layer.d), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.vc = torch.full_like(self.kc, float("nan"))
        self.lens, self.held, self.count = i32([0] * B), i32([0] * B), i32([pages])
        self.free = torch.randperm(pages, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
        self.bt = i32([[-1] * (pages // B + 1)] * B)
        self.ws = torch.empty(256, dtype=torch.uint8, device="cuda")

    def plan(self, new, n, parents=None, max_tree=0, buffers=None):
        out = (buffers or ola.orthros_plan_step_buffers(self.B, n, max_tree))._replace(pages_held=self.held, free_count=self.count)
        return ola.orthros_plan_step(self.lens, new, self.held, self.free, self.count, self.bt, self.page, n, parents=parents,
                                     max_tree=max_tree, out=out, workspace=self.ws)

    def chunk(self, x):
        """Consecutive tokens x[b] [m, D_MODEL] of every sequence, m >= 1; (o_base rows, o_out of the last ones)."""
        new = [t.shape[0] for t in x]
        p = self.plan(i32(new), sum(new))
        rows = torch.cat(list(x) + [t[-1:] for t in x])
        o = self.layer.step(rows, sum(new), self.kc, self.vc, self.bt, p.token_seq, p.token_pos, p.q_indptr, p.kv_lens,
                            torch.arange(self.B + 1, dtype=torch.int32, device="cuda"), p.kv_lens - 1, max(new),
                            token_slots=p.token_slots)
        assert self.layer.check() == (0, 0) and ola.orthros_check(self.ws) == (0, 0)
        self.lens.copy_(p.cache_lens)
        return o

    def rows(self, b):
        n = int(self.lens[b])
        at = torch.arange(n, device="cuda")
        slots = self.bt[b, at // self.page].long() * self.page + at % self.page
        return self.kc.flatten(0, 1)[slots], self.vc.flatten(0, 1)[slots]


def draft(r, n):
    return [-1 if i == 0 else r.randint(-1, i - 1) for i in range(n)]


def path_to(tree, i):
    out = [i]
    while tree[out[0]] >= 0:
        out.insert(0, tree[out[0]])
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("normed", [True, False])
@pytest.mark.parametrize("Hq,Hkv,d,window,layout,page", [(8, 2, 128, 100, "half", 16), (32, 8, 128, 7, "interleaved", 64),
                                                         (4, 4, 64, 64, "half", 24)])
def test_trees_agree_with_their_paths(Hq, Hkv, d, window, layout, page, normed):
    layer, g = make_layer(Hq, Hkv, d, window, layout, seed=Hq, normed=normed)
    r, B = random.Random(Hq), 3
    pages = B * (300 // page + 2)
    prompt = [torch.randn(m, D_MODEL, generator=g).bfloat16().cuda() for m in (150, 33, 1)]
    srv = Server(layer, B, page, pages)
    srv.chunk(prompt)
    said = list(prompt)  # what each sequence consists of
    for sizes in ((20, 9, 33), (1, 30, 2)):
        trees = [draft(r, m) for m in sizes]
        x = [torch.randn(m, D_MODEL, generator=g).bfloat16().cuda() for m in sizes]
        n, pad = sum(sizes), 11
        first = np.concatenate([[0], np.cumsum(sizes)])
        p = srv.plan(i32(sizes), n + pad, i32([q for t in trees for q in t] + [0] * pad), max_tree=33)
        rows = torch.cat(x + [torch.zeros(pad, D_MODEL, dtype=torch.bfloat16, device="cuda")])
        ob, oo = layer.tree_step(torch.cat([rows, rows]), p, srv.kc, srv.vc, srv.bt, max(sizes))
        assert layer.check() == (0, 0) and ola.orthros_check(srv.ws) == (0, 0)
        # some tokens of each tree, as the end of their path behind the same prompt
        ends = [[r.randrange(m) for m in sizes] for _ in range(4)] + [[m - 1 for m in sizes]]
        for at in ends:
            paths = [path_to(t, i) for t, i in zip(trees, at)]
            line = Server(layer, B, page, pages)
            line.chunk(said)
            lb, lo = line.chunk([t[q] for t, q in zip(x, paths)])
            last = np.cumsum([len(q) for q in paths]) - 1
            node = [int(first[b]) + at[b] for b in range(B)]
            assert float((ob[node].float() - lb[last].float()).abs().max()) <= 4e-2
            assert float((oo[node].float() - lo.float()).abs().max()) <= 4e-2
        # the last of those paths is accepted, of the first sequence none of it
        paths[0] = []
        most = max(map(len, paths)) + 1
        cws = torch.empty(256, dtype=torch.uint8, device="cuda")
        ola.orthros_tree_commit(srv.kc, srv.vc, srv.bt, p.q_indptr, p.kv_lens, i32([q + [0] * (most - len(q)) for q in paths]),
                                i32([len(q) for q in paths]), out=srv.lens, workspace=cws)
        assert ola.orthros_check(cws) == (0, 0)
        said = [torch.cat([s, t[q]]) for s, t, q in zip(said, x, paths)]
        assert srv.lens.tolist() == [s.shape[0] for s in said]
        line = Server(layer, B, page, pages)
        line.chunk(said)
        for b in range(B):
            for a, w in zip(srv.rows(b), line.rows(b)):
                assert bool(((a.float() - w.float()).abs() <= 2.0 ** -7 * w.float().abs() + 1e-6).all())
    # and the sequences go on by single tokens
    x = [torch.randn(1, D_MODEL, generator=g).bfloat16().cuda() for _ in range(B)]
    got, want = srv.chunk(x), line.chunk(x)
    assert all(float((a.float() - b.float()).abs().max()) <= 4e-2 for a, b in zip(got, want))


@pytest.mark.gpu
def test_a_captured_cycle_follows_its_inputs():
    """Plan, tree step and commit in one graph: replays give the eager calls' bits as lengths grow."""
    B, page, n, most, max_tree = 4, 16, 60, 5, 16
    layer, g = make_layer(8, 2, 128, 50, "half", seed=5, normed=True)
    pages = 40
    eager, graphed = Server(layer, B, page, pages), Server(layer, B, page, pages)
    prompt = [torch.randn(m, D_MODEL, generator=g).bfloat16().cuda() for m in (40, 3, 70, 16)]
    eager.chunk(prompt), graphed.chunk(prompt)
    x = torch.empty(2 * n, D_MODEL, dtype=torch.bfloat16, device="cuda")
    new, parents, acc, cnt = i32([1] * B), i32([0] * n), i32([[0] * most] * B), i32([0] * B)

    def cycle(srv, buffers, ws, cws):
        p = srv.plan(new, n, parents, max_tree, buffers)
        o = layer.tree_step(x, p, srv.kc, srv.vc, srv.bt, max_tree, ws)
        ola.orthros_tree_commit(srv.kc, srv.vc, srv.bt, p.q_indptr, p.kv_lens, acc, cnt, out=srv.lens, workspace=cws)
        return o, p

    args = [(ola.orthros_plan_step_buffers(B, n, max_tree), layer.tree_workspaces(B, n, max_tree, eager.bt.shape[1], page),
             torch.empty(256, dtype=torch.uint8, device="cuda")) for _ in range(2)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        (gb, go), _ = cycle(graphed, *args[1])
    r = random.Random(3)
    for _ in range(6):
        sizes = [r.randint(0, max_tree - 2) for _ in range(B)]
        trees = [draft(r, m) for m in sizes]
        flat = [q for t in trees for q in t]
        paths = [path_to(t, r.randrange(len(t)))[:most] if t else [] for t in trees]
        new.copy_(i32(sizes))
        parents.copy_(i32(flat + [0] * (n - len(flat))))
        acc.copy_(i32([q + [0] * (most - len(q)) for q in paths]))
        cnt.copy_(i32([len(q) for q in paths]))
        x.copy_(torch.randn(2 * n, D_MODEL, generator=g))
        (eb, eo), p = cycle(eager, *args[0])
        graph.replay()
        m = sum(sizes)
        assert torch.equal(eb[:m], gb[:m]) and torch.equal(eo[:m], go[:m])
        assert torch.equal(eager.lens, graphed.lens) and torch.equal(eager.bt, graphed.bt) and torch.equal(eager.count, graphed.count)
        assert all(ola.orthros_check(w) == (0, 0) for w in (graphed.ws, args[1][2], *args[1][1]))
        for b in range(B):
            assert all(torch.equal(s, t) for s, t in zip(eager.rows(b), graphed.rows(b)))


@pytest.mark.gpu
def test_a_sequence_without_pages_keeps_its_state():
    """One sequence finds no page: its rows are NaN, its length and cache stay, the others' step is good;
    when another ends, it goes on."""
    layer, g = make_layer(4, 2, 64, 1000, "half", seed=6, normed=True)
    B, page = 3, 8
    srv = Server(layer, B, page, 9)
    srv.chunk([torch.randn(m, D_MODEL, generator=g).bfloat16().cuda() for m in (16, 30, 17)])  # 2 + 4 + 3 pages
    sizes, n = [3, 2, 4], 9
    rows = torch.randn(n, D_MODEL, generator=g).bfloat16().cuda()
    parents = i32([-1, 0, 0, -1, 0, -1, 0, 1, 1])
    before = [t.clone() for t in srv.rows(0)]
    p = srv.plan(i32(sizes), n, parents, 4)
    assert ola.orthros_check(srv.ws)[1] == 32
    ob, oo = layer.tree_step(torch.cat([rows, rows]), p, srv.kc, srv.vc, srv.bt, 4)
    assert layer.check() == (5, 4)  # the attention: no place in the step
    assert bool(torch.isnan(ob[:3]).all()) and bool(torch.isnan(oo[:3]).all())
    assert bool(torch.isfinite(ob[3:]).all()) and bool(torch.isfinite(oo[3:]).all())
    cws = torch.empty(256, dtype=torch.uint8, device="cuda")
    ola.orthros_tree_commit(srv.kc, srv.vc, srv.bt, p.q_indptr, p.kv_lens, i32([[0, 1]] * 3), i32([2, 1, 2]), out=srv.lens,
                            workspace=cws)
    assert ola.orthros_check(cws)[1] == 4 and srv.lens.tolist() == [16, 31, 19] and srv.held.tolist() == [2, 4, 3]
    assert all(torch.equal(a, b) for a, b in zip(before, srv.rows(0)))
    # the second sequence ends; the first takes one of its pages
    p = srv.plan(i32([3, -1, 0]), 3, parents[:3], 4)
    srv.lens.copy_(p.cache_lens)
    assert ola.orthros_check(srv.ws) == (0, 0) and srv.held.tolist() == [3, 0, 3] and srv.count.tolist() == [3]
    assert srv.lens.tolist() == [19, 0, 19]


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_training_gradients_with_norms_against_autograd(layout):
    Hq, Hkv, d, T, B, window, rot = 4, 2, 64, 90, 2, 30, 48
    layer, g = make_layer(Hq, Hkv, d, window, layout, seed=3, normed=True, rot=rot)
    q, k, v = (torch.randn(B, T, h, d, generator=g).bfloat16().cuda() for h in (Hq, Hkv, Hkv))
    indptr = np.array([0, 3, 5], dtype=np.int32)
    opos = torch.tensor([10, 89, 10, 0, 50], dtype=torch.int32, device="cuda")
    (ob, oo), saved = layer.forward(q, k, v, indptr, opos)
    db, do = torch.randn(ob.shape, generator=g).bfloat16().cuda(), torch.randn(oo.shape, generator=g).bfloat16().cuda()
    got = layer.backward(saved, db, do)
    assert layer.check() == (0, 0)

    names = ("q", "k", "v", "alpha_base", "beta_base", "alpha_out", "beta_out", "q_norm", "k_norm")
    leaves = {n: t.double().detach().clone().requires_grad_() for n, t in
              zip(names, (q, k, v, *layer.affines, layer.q_norm, layer.k_norm))}
    th = torch.arange(T, device="cuda").double()[:, None] * layer.freq.cuda()
    ia, ib = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half" else (slice(0, rot, 2), slice(1, rot, 2))

    def rot_(u, c, s):
        y = u.clone()
        y[..., ia] = u[..., ia] * c[:, None] - u[..., ib] * s[:, None]
        y[..., ib] = u[..., ia] * s[:, None] + u[..., ib] * c[:, None]
        return y

    def norm(x, w):
        return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + layer.norm_eps) * w

    c, s = torch.cos(th), torch.sin(th)
    kr = rot_(norm(leaves["k"], leaves["k_norm"]), c, s).repeat_interleave(Hq // Hkv, 2)
    vv = leaves["v"].repeat_interleave(Hq // Hkv, 2)
    t = torch.arange(T, device="cuda")
    band = (t[None, :] <= t[:, None]) & (t[None, :] > t[:, None] - window)
    nq = norm(leaves["q"], leaves["q_norm"])
    qr = rot_(nq * leaves["alpha_base"] + leaves["beta_base"], c, s)
    z = torch.einsum("bthd,bjhd->bhtj", qr, kr) * d ** -0.5
    o = torch.einsum("bhtj,bjhd->bthd", torch.softmax(z.masked_fill(~band, float("-inf")), -1), vv)
    seq, p = torch.tensor([0, 0, 0, 1, 1], device="cuda"), opos.long()
    qo = rot_(nq[seq, p] * leaves["alpha_out"] + leaves["beta_out"], c[p], s[p])
    z = torch.einsum("nhd,njhd->nhj", qo, kr[seq]) * d ** -0.5
    z = z.masked_fill(t[None, None, :] > p[:, None, None], float("-inf"))
    oo64 = torch.einsum("nhj,njhd->nhd", torch.softmax(z, -1), vv[seq])
    assert float((ob.double() - o.detach()).abs().max()) <= 3e-2 and float((oo.double() - oo64.detach()).abs().max()) <= 3e-2
    ((o * db.double()).sum() + (oo64 * do.double()).sum()).backward()
    rms = float(db.float().pow(2).mean().sqrt())
    rows = dict(alpha_base=B * T, beta_base=B * T, alpha_out=5, beta_out=5, q_norm=B * T * Hq, k_norm=B * T * Hkv)
    for n, leaf in leaves.items():
        ref, a = leaf.grad, got["d" + n if n in "qkv" else "d_" + n].double()
        floor = rms * rows.get(n, 1) ** 0.5
        err = float(((a - ref).abs() / (ref.pow(2).mean().sqrt() + ref.abs() + floor)).max())
        assert err <= 5e-2, (n, err)


@pytest.mark.gpu
def test_refusals():
    layer, g = make_layer(4, 2, 64, 30, "half", seed=1, normed=True)
    srv = Server(layer, 1, 8, 4)
    x = torch.randn(2, D_MODEL, generator=g).bfloat16().cuda()
    with pytest.raises(ValueError):  # norms need slots
        layer.step(x, 1, srv.kc, srv.vc, srv.bt, i32([0]), i32([0]), i32([0, 1]), i32([1]), i32([0, 1]), i32([0]), 1)
    p = srv.plan(i32([1]), 1, i32([-1]), 1)
    with pytest.raises(ValueError):
        layer.tree_step(x[:1], p, srv.kc, srv.vc, srv.bt, 1)
    with pytest.raises(ValueError):
        RotaryLayer(layer.w_qkv, layer.affines, layer.freq, 4, 2, 64, 30, q_norm=layer.q_norm)


@pytest.mark.gpu
def test_two_batches_at_once():
    """Cycles of two batches on two streams, with workspaces of their own, give the bits of one after the other."""
    B, page, n, max_tree, most = 6, 16, 90, 20, 4
    layer, g = make_layer(8, 2, 128, 60, "interleaved", seed=7, normed=True)
    r = random.Random(5)
    rounds = []
    for _ in range(8):
        sizes = [r.randint(1, max_tree - 5) for _ in range(B)]
        trees = [draft(r, m) for m in sizes]
        flat = [q for t in trees for q in t]
        paths = [path_to(t, r.randrange(len(t)))[:most] for t in trees]
        rounds.append((i32(sizes), i32(flat + [0] * (n - len(flat))), i32([q + [0] * (most - len(q)) for q in paths]),
                       i32([len(q) for q in paths]), torch.randn(2 * n, D_MODEL, generator=g).bfloat16().cuda(), sum(sizes)))
    prompts = [[torch.randn(m, D_MODEL, generator=g).bfloat16().cuda() for m in ms] for ms in ((9, 200, 33, 1, 64, 300), (5, 1, 500, 2, 16, 17))]

    def start():
        out = []
        for p in prompts:
            out.append(Server(layer, B, page, 200))
            out[-1].chunk(p)
        torch.cuda.synchronize()
        return out

    def cycle(srv, rnd, cws):
        new, parents, acc, cnt, x, m = rnd
        p = srv.plan(new, n, parents, max_tree)
        o = layer.tree_step(x, p, srv.kc, srv.vc, srv.bt, max_tree)
        ola.orthros_tree_commit(srv.kc, srv.vc, srv.bt, p.q_indptr, p.kv_lens, acc, cnt, out=srv.lens, workspace=cws)
        return [t[:m].clone() for t in o]

    cws = [torch.empty(256, dtype=torch.uint8, device="cuda") for _ in range(2)]
    want = []
    for i, srv in enumerate(start()):
        want.append([cycle(srv, rounds[(k + 3 * i) % 8], cws[i]) for k in range(8)])
    servers = start()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for k in range(8):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(cycle(servers[i], rounds[(k + 3 * i) % 8], cws[i]))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for s, t in zip(a, b) for x, y in zip(s, t))
    assert all(ola.orthros_check(w) == (0, 0) for w in (*cws, *(s.ws for s in servers)))
