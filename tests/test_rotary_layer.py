"""The rotary layer (projection, rotated append, attention over the cache; rotation around
prefill and its backward): serving a prompt in chunks and then token by token agrees with
the training forward over the whole sequence, and the gradients with autograd in fp64.

Outputs: both paths read the same bf16 queries, keys and values and each lies within the
attention contract (2e-2 absolute for N(0, 1) inputs) of the exact value. Gradients: the
prefill backward's own bound (5e-2 of rms(ref) + |ref| + floor), whose terms the orthogonal
rotation does not enlarge; the floor is rms(dO), times sqrt(rows summed) for the affines.
"""
import numpy as np
import pytest
import torch

import efficient_long_context_gb300 as ola
from efficient_long_context_gb300.rotary_layer import RotaryLayer

pytestmark = pytest.mark.gpu


def make_layer(Hq, Hkv, d, window, layout, seed, d_model=256, rot=None):
    g = torch.Generator().manual_seed(seed)
    w = (torch.randn((Hq + 2 * Hkv) * d, d_model, generator=g) / d_model ** 0.5).bfloat16().cuda()
    aff = []
    for _ in range(2):
        aff += [(1 + 0.1 * torch.randn(Hq, d, generator=g)).cuda(), (0.1 * torch.randn(Hq, d, generator=g)).cuda()]
    freq, amp = ola.orthros_rotary_frequencies(rot or d, 10000.0, "bands_tempered", factor=4.0, original_length=4096.0)
    return RotaryLayer(w, aff, freq, Hq, Hkv, d, window, layout, amp), g


@pytest.mark.parametrize("Hq,Hkv,d,window,layout,page", [(8, 2, 128, 100, "half", 16), (32, 8, 128, 300, "interleaved", 64),
                                                         (4, 4, 64, 64, "half", 24)])
def test_serving_in_chunks_and_steps_matches_one_prefill(Hq, Hkv, d, window, layout, page):
    layer, g = make_layer(Hq, Hkv, d, window, layout, seed=Hq)
    B, T = 3, 330
    x = torch.randn(B, T, 256, generator=g).bfloat16().cuda()
    mp = (T + page - 1) // page
    bt = torch.randperm(B * mp, generator=g).to(torch.int32).view(B, mp).cuda()
    kc = torch.full((B * mp, page, Hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    vc = torch.full_like(kc, float("nan"))
    # sequences advance by chunks of their own, then by single tokens; sequence 2 sits one step out
    plan = [(200, 70, 130), (100, 129, 0), (1, 1, 1), (1, 1, 64), (1, 1, 1)]
    at = [0] * B
    base = torch.zeros(B, T, Hq, d, device="cuda")
    outs = []
    for new in plan:
        seq = [b for b in range(B) for _ in range(new[b])]
        pos = [at[b] + i for b in range(B) for i in range(new[b])]
        at = [a + n for a, n in zip(at, new)]
        live = [b for b in range(B) if new[b]]
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
        rows = torch.cat([x[seq, pos], x[live, [at[b] - 1 for b in live]]])
        ob, oo = layer.step(rows, len(seq), kc, vc, bt, i32(seq), i32(pos), i32(np.concatenate([[0], np.cumsum(new)])),
                            i32(at), i32(np.concatenate([[0], np.cumsum([int(n > 0) for n in new])])),
                            i32([at[b] - 1 for b in live]), max(new))
        base[seq, pos] = ob.float()
        outs += [(b, at[b] - 1, oo[i].float()) for i, b in enumerate(live)]
    # the same tokens in one training forward: raw projections, output rows at the served positions
    one = [torch.ones(Hq, d, device="cuda"), torch.zeros(Hq, d, device="cuda")] * 2
    q, _, k, v = ola.orthros_qkv_project(x.flatten(0, 1), B * T, layer.w_qkv, Hq, Hkv, d, *one, kv_out=True)
    outs.sort(key=lambda o: (o[0], o[1]))
    indptr = np.concatenate([[0], np.cumsum([sum(o[0] == b for o in outs) for b in range(B)])]).astype(np.int32)
    (ob, oo), _ = layer.forward(q.view(B, T, Hq, d), k.view(B, T, Hkv, d), v.view(B, T, Hkv, d), indptr,
                                torch.tensor([o[1] for o in outs], dtype=torch.int32, device="cuda"))
    for b in range(B):
        # the raw projection is rounded before its affine here and after it in step(): one bf16
        # rounding of q apart (2^-8 per logit of a few units), besides the two contracts
        assert float((base[b, :at[b]] - ob[b, :at[b]].float()).abs().max()) <= 6e-2
    assert float((torch.stack([o[2] for o in outs]) - oo.float()).abs().max()) <= 6e-2


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_training_gradients_against_autograd(layout):
    Hq, Hkv, d, T, B, window, rot = 4, 2, 64, 90, 2, 30, 48
    layer, g = make_layer(Hq, Hkv, d, window, layout, seed=3, rot=rot)
    q, k, v = (torch.randn(B, T, h, d, generator=g).bfloat16().cuda() for h in (Hq, Hkv, Hkv))
    indptr = np.array([0, 3, 5], dtype=np.int32)
    opos = torch.tensor([10, 89, 10, 0, 50], dtype=torch.int32, device="cuda")
    (ob, oo), saved = layer.forward(q, k, v, indptr, opos)
    db, do = torch.randn(ob.shape, generator=g).bfloat16().cuda(), torch.randn(oo.shape, generator=g).bfloat16().cuda()
    got = layer.backward(saved, db, do)

    leaves = {n: t.double().detach().clone().requires_grad_() for n, t in
              zip(("q", "k", "v", "alpha_base", "beta_base", "alpha_out", "beta_out"), (q, k, v, *layer.affines))}
    th = torch.arange(T, device="cuda").double()[:, None] * layer.freq.cuda()
    ia, ib = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half" else (slice(0, rot, 2), slice(1, rot, 2))

    def rot_(u, c, s):  # u [..., n, H, d], c, s [n, pairs]
        y = u.clone()
        y[..., ia] = layer.amplitude * (u[..., ia] * c[:, None] - u[..., ib] * s[:, None])
        y[..., ib] = layer.amplitude * (u[..., ia] * s[:, None] + u[..., ib] * c[:, None])
        return y

    c, s = torch.cos(th), torch.sin(th)
    kr = rot_(leaves["k"], c, s).repeat_interleave(Hq // Hkv, 2)
    vv = leaves["v"].repeat_interleave(Hq // Hkv, 2)
    t = torch.arange(T, device="cuda")
    band = (t[None, :] <= t[:, None]) & (t[None, :] > t[:, None] - window)
    qr = rot_(leaves["q"] * leaves["alpha_base"] + leaves["beta_base"], c, s)
    z = torch.einsum("bthd,bjhd->bhtj", qr, kr) * d ** -0.5
    o = torch.einsum("bhtj,bjhd->bthd", torch.softmax(z.masked_fill(~band, float("-inf")), -1), vv)
    seq = torch.tensor([0, 0, 0, 1, 1], device="cuda")
    p = opos.long()
    qo = rot_((leaves["q"][seq, p] * leaves["alpha_out"] + leaves["beta_out"]), c[p], s[p])
    z = torch.einsum("nhd,njhd->nhj", qo, kr[seq]) * d ** -0.5
    z = z.masked_fill(t[None, None, :] > p[:, None, None], float("-inf"))
    oo64 = torch.einsum("nhj,njhd->nhd", torch.softmax(z, -1), vv[seq])
    assert float((ob.double() - o.detach()).abs().max()) <= 3e-2 and float((oo.double() - oo64.detach()).abs().max()) <= 3e-2
    ((o * db.double()).sum() + (oo64 * do.double()).sum()).backward()
    rms = float(db.float().pow(2).mean().sqrt())
    for n, leaf in leaves.items():
        ref, a = leaf.grad, got["d" + n if n in "qkv" else "d_" + n].double()
        floor = rms if n in "qkv" else rms * (B * T if n.endswith("base") else 5) ** 0.5
        err = float(((a - ref).abs() / (ref.pow(2).mean().sqrt() + ref.abs() + floor)).max())
        assert err <= 5e-2, (n, err)


def test_output_positions_outside_their_sequence():
    """A position outside [0, T) gives a NaN row and no gradient: the gradients are those of the other
    rows alone, in its neighbours' sequences too."""
    Hq, Hkv, d, T, B, window = 4, 2, 64, 90, 3, 30
    layer, g = make_layer(Hq, Hkv, d, window, "half", seed=5)
    q, k, v = (torch.randn(B, T, h, d, generator=g).bfloat16().cuda() for h in (Hq, Hkv, Hkv))
    db = torch.randn(B, T, Hq, d, generator=g).bfloat16().cuda()
    good = [(0, 10), (0, 89), (1, 10), (2, 50)]
    do = torch.randn(len(good), Hq, d, generator=g).bfloat16().cuda()

    def run(rows, do_rows):
        indptr = np.concatenate([[0], np.cumsum([sum(r[0] == b for r in rows) for b in range(B)])]).astype(np.int32)
        (ob, oo), saved = layer.forward(q, k, v, indptr, torch.tensor([r[1] for r in rows], dtype=torch.int32, device="cuda"))
        return ob, oo, layer.backward(saved, db, do_rows)

    ob, oo, want = run(good, do)
    for where, bad in ((0, (0, -1)), (2, (0, T)), (4, (2, 1 << 30)), (2, (1, -(2 ** 31))), (3, (2, 2 ** 31 - 1))):
        rows = good[:where] + [bad] + good[where:]
        keep = [i for i in range(len(rows)) if i != where]
        do_rows = torch.cat([do[:where], torch.full_like(do[:1], 100.0), do[where:]])
        ob2, oo2, got = run(rows, do_rows)
        assert torch.equal(ob2, ob) and float((oo2[keep].float() - oo.float()).abs().max()) <= 2e-2
        assert bool(torch.isnan(oo2[where]).all())
        for n in want:
            # the same terms, each rounded to bf16 at most three times (2^-8 each) before the fp32 sums;
            # the bad row's 100s would move every sum they enter by more than this
            a, b = got[n].double(), want[n].double()
            assert bool(((a - b).abs() <= 2.0 ** -6 * (b.abs() + b.abs().max())).all()), (bad, n)


def test_output_rows_counted_on_the_gpu():
    """out_indptr may be a GPU tensor, as orthros_prefill takes it."""
    layer, g = make_layer(4, 2, 64, 30, "half", seed=7)
    q, k, v = (torch.randn(2, 50, h, 64, generator=g).bfloat16().cuda() for h in (4, 2, 2))
    opos = torch.tensor([10, 49, 0], dtype=torch.int32, device="cuda")
    host = layer.forward(q, k, v, np.array([0, 2, 3], dtype=np.int32), opos)
    dev = layer.forward(q, k, v, torch.tensor([0, 2, 3], dtype=torch.int32, device="cuda"), opos)
    for a, b in zip(host[0], dev[0]):
        assert torch.equal(a, b)
    grads = [layer.backward(s, torch.ones_like(q), torch.ones_like(o[1])) for o, s in (host, dev)]
    assert torch.equal(grads[0]["dv"], grads[1]["dv"])


def test_repeated_output_positions_add_in_a_fixed_order():
    """fp32, hundreds of output rows at one position: the same backward gives the same bits of dq, which
    holds the sum of the rows' gradients (at most 500 fp32 additions of 2^-24 each)."""
    Hq, Hkv, d, T, B, window = 4, 2, 64, 40, 2, 30
    layer, g = make_layer(Hq, Hkv, d, window, "half", seed=6)
    q, k, v = (torch.randn(B, T, h, d, generator=g).cuda() for h in (Hq, Hkv, Hkv))
    pos = [7] * 400 + [39, 3] + [7] * 98 + [39] * 200 + [0]
    indptr, opos = np.array([0, 500, 701], dtype=np.int32), torch.tensor(pos, dtype=torch.int32, device="cuda")
    (ob, oo), saved = layer.forward(q, k, v, indptr, opos)
    db, do = torch.randn(ob.shape, generator=g).cuda(), torch.randn(oo.shape, generator=g).cuda()
    got = layer.backward(saved, db, do)["dq"]
    for _ in range(5):
        assert torch.equal(layer.backward(saved, db, do)["dq"], got)
    qf, q_sel, _, tok, qr, kr, _, qo, _, _, out = saved
    grads = ola.orthros_prefill_backward(qr, kr, v, *layer.identity, *layer.identity, indptr, opos, window, None, *out, db, do,
                                         q_out=qo)
    rope = dict(layout=layer.layout, amplitude=layer.amplitude)
    base, _, _ = ola.orthros_rotate_backward(grads["dq"].flatten(0, 1), qf, tok, layer.steps, alpha=layer.affines[0], **rope)
    sel, _, _ = ola.orthros_rotate_backward(grads["dq_out"], q_sel, opos, layer.steps, alpha=layer.affines[2], **rope)
    rows = torch.repeat_interleave(torch.arange(B), torch.tensor([500, 201])).cuda() * T + opos
    want = base.double().index_add_(0, rows, sel.double())
    mag = base.double().abs().index_add_(0, rows, sel.double().abs())
    assert bool(((got.flatten(0, 1).double() - want).abs() <= 500 * 2.0 ** -24 * mag).all())


def test_check_reports_what_the_calls_of_a_step_found():
    """A position, page or length that does not exist skips a cache write or makes rows NaN; check() and
    the caller's own workspaces tell, and a good step after it is clean again."""
    Hq, Hkv, d, page = 8, 2, 128, 16
    layer, g = make_layer(Hq, Hkv, d, 100, "half", seed=8)
    assert layer.check() == (0, 0)  # no call yet
    x = torch.randn(5 + 2, 256, generator=g).bfloat16().cuda()
    bt = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device="cuda")
    kc = torch.zeros((4, page, Hkv, d), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    good = dict(block_table=bt, token_seq=i32(0, 0, 0, 1, 1), token_pos=i32(0, 1, 2, 0, 1), new_indptr=i32(0, 3, 5),
                kv_lens=i32(3, 2), out_indptr=i32(0, 1, 2), out_positions=i32(2, 1), max_new=3)
    own = layer.step_workspaces(2, 5, 2, 3, 2, page)
    clean = layer.step(x, 5, kc, vc, **good)
    assert layer.check() == (0, 0)
    for ws in (None, own):
        for bad, bits in ((dict(token_pos=i32(0, 1, 2, 0, 2 * page)), 1), (dict(token_seq=i32(0, 0, 0, 1, 2)), 1),
                          (dict(block_table=i32(0, 1, 4, 3).view(2, 2)), 2), (dict(kv_lens=i32(3, 2 * page + 1)), 4),
                          (dict(max_new=2), 4)):
            layer.step(x, 5, kc, vc, **dict(good, **bad), workspaces=ws)
            assert layer.check() == (5, bits), bad
            if ws is not None:
                assert max(ola.orthros_check(w)[1] for w in ws) == bits
            again = layer.step(x, 5, kc, vc, **good, workspaces=ws)
            assert layer.check() == (0, 0)
            assert all(torch.equal(a, b) for a, b in zip(again, clean))


def test_check_reports_what_training_found():
    layer, g = make_layer(4, 2, 64, 30, "half", seed=9)
    q, k, v = (torch.randn(2, 50, h, 64, generator=g).bfloat16().cuda() for h in (4, 2, 2))
    for pos, want in ((49, (0, 0)), (50, (5, 1)), (-1, (5, 1))):
        opos = torch.tensor([10, pos, 0], dtype=torch.int32, device="cuda")
        (_, oo), saved = layer.forward(q, k, v, np.array([0, 2, 3], dtype=np.int32), opos)
        assert layer.check() == want
        layer.backward(saved, torch.ones_like(q), torch.ones_like(oo))
        assert layer.check() == want


def test_step_in_a_graph_reports_after_a_replay():
    """A captured step's check() reads what the last replay left."""
    layer, g = make_layer(4, 2, 64, 30, "half", seed=10)
    x = torch.randn(2, 256, generator=g).bfloat16().cuda()
    bt = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    kc = torch.zeros((2, 16, 2, 64), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    pos, lens, args = i32(0), i32(1), dict(new_indptr=i32(0, 1), out_indptr=i32(0, 1), token_seq=i32(0), max_new=1)
    ws = layer.step_workspaces(1, 1, 1, 1, 2, 16)

    def step():
        return layer.step(x, 1, kc, vc, bt, args["token_seq"], pos, args["new_indptr"], lens, args["out_indptr"], pos, 1,
                          workspaces=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t, want in ((0, (0, 0)), (31, (0, 0)), (32, (5, 5)), (5, (0, 0))):
        pos.fill_(t)
        lens.fill_(t + 1)
        graph.replay()
        assert layer.check() == want, t
