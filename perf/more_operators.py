"""A serving step with drafted trees, and normed queries and keys: the calls,
their plain forms and their exact values.

Operators of a layer whose queries and keys are normed per head, and of a step
that drafts a tree of tokens for each sequence and verifies it in one pass:

norm_rotate       y = m R(t) (alpha (.) (w (.) x / rms(x)) + beta): the norm of
                  a head, the stream's affine and the rotary position.
norm_backward     dx, d_w, d_alpha, d_beta of the same.
norm_append       new keys normed, rotated and written with their values to the
                  slots that the plan gave them; both query streams likewise.
plan              what a step needs from its lengths, built on the GPU: pages
                  taken from the free list into the block tables, sequence,
                  position and slot of every token, the ancestor masks of trees.
tree_attend       the drafted tokens over the paged cache: every cached key
                  before the tree (in the window), and the token's ancestors.
commit            the accepted path's keys and values moved to the places they
                  have in the sequence, in every layer's cache.

`own = False` computes them with elementary torch operations in 32 bits
(angles in 64); `own = True` calls the library.
"""
from __future__ import annotations

import math
import random

import torch

own = False

# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
# Head shapes are the repository's: GQA 32/8 with d = 128 (its 128K prefill,
# fine-tuning and decoding workloads), 16 heads with d = 128 (pre-training),
# 4 heads with d = 64 (the small fp32 workload).


def listed():
    return [
        # both queries of 32 decoding pairs at far positions: launch latency counts
        dict(name="norm_rotate_decode_64", op="norm_rotate", n=64, H=32, d=128, rot=128, layout="half", affine=True,
             dtype="bf16", pos="far"),
        # the queries of a fine-tuning step, 4 x 8192 tokens
        dict(name="norm_rotate_sft_32768", op="norm_rotate", n=32768, H=32, d=128, rot=128, layout="interleaved",
             affine=True, dtype="bf16", pos="seq"),
        # gradient of a small fp32 model's keys, odd length, half of the head rotated, no affine
        dict(name="norm_grad_f32_2049", op="norm_backward", n=2049, H=4, d=64, rot=32, layout="interleaved",
             affine=False, dtype="f32", pos="seq"),
        # gradient of the fine-tuning queries, with the norm's weight and the affine
        dict(name="norm_grad_sft_32768", op="norm_backward", n=32768, H=32, d=128, rot=128, layout="half",
             affine=True, dtype="bf16", pos="seq"),
        # drafted trees of 1 to 24 tokens of 32 sequences, both query streams
        dict(name="norm_append_trees_32", op="norm_append", B=32, new_lo=1, new_hi=24, hist=2048, both=True, Hq=32,
             Hkv=8, d=128, rot=128, layout="half", affine=True, dtype="bf16", page=64, sizes=21),
        # prompts of five sequences, about 8000 tokens, small pages
        dict(name="norm_append_prompts_5", op="norm_append", B=5, new_lo=900, new_hi=2300, hist=4096, both=False, Hq=32,
             Hkv=8, d=128, rot=64, layout="interleaved", affine=False, dtype="bf16", page=16, sizes=22),
        # 64 sequences decode one token each; a few take a new page
        dict(name="plan_decode_64", op="plan", B=64, tree=False, new_lo=1, new_hi=1, hist=30000, page=64, pad=0,
             sizes=23),
        # 500 sequences draft trees of up to 64 tokens into small pages, some sequences end, rows to spare
        dict(name="plan_trees_500", op="plan", B=500, tree=True, new_lo=1, new_hi=64, hist=8000, page=16, pad=2000,
             sizes=24),
        # one user, a tree of 25 tokens, 32K of history: latency and the split of the key axis
        dict(name="tree_one_32k", op="tree_attend", B=1, new_lo=25, new_hi=25, hist_lo=32743, hist_hi=32743, Hq=32,
             Hkv=8, d=128, window=0, page=64, sizes=25),
        # 32 sequences verify trees of 9 to 60 tokens over 4K-20K of history, small pages
        dict(name="tree_batch_32", op="tree_attend", B=32, new_lo=9, new_hi=60, hist_lo=4096, hist_hi=20000, Hq=32,
             Hkv=8, d=128, window=0, page=16, sizes=26),
        # the accepted tokens of 32 sequences in one layer's cache
        dict(name="commit_32", op="commit", B=32, layers=1, new_lo=8, new_hi=32, most=6, hist=2000, Hkv=8, d=128,
             dtype="bf16", page=64, sizes=27),
        # the same in all 32 layers of a model at once
        dict(name="commit_32_layers", op="commit", B=48, layers=32, new_lo=8, new_hi=60, most=8, hist=300, Hkv=8, d=128,
             dtype="bf16", page=16, sizes=28),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rotate", "norm_backward", "norm_append", "plan", "tree_attend", "tree_attend", "commit"])
    d = rng.choice([64, 128, 128])
    Hq, Hkv = rng.choice([(32, 8), (32, 8), (16, 16), (4, 4), (8, 2), (12, 4)])
    layout = rng.choice(["half", "interleaved"])
    rot = rng.choice([r for r in (16, 32, 48, 64, 96, 128) if r <= d])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    page = rng.choice([8, 16, 32, 48, 64, 128])
    sizes = rng.randint(0, 99999)
    if op in ("norm_rotate", "norm_backward"):
        return dict(op=op, n=_log_int(rng, 1, 32768 if dtype == "bf16" else 16384), H=rng.choice([Hq, Hkv]), d=d,
                    rot=rot, layout=layout, affine=rng.random() < 0.5, dtype=dtype, pos=rng.choice(["seq", "far"]))
    if op == "norm_append":
        if rng.random() < 0.6:
            return dict(op=op, B=_log_int(rng, 1, 64), new_lo=1, new_hi=_log_int(rng, 1, 64), hist=2048,
                        both=rng.random() < 0.7, Hq=Hq, Hkv=Hkv, d=d, rot=rot, layout=layout, affine=rng.random() < 0.5,
                        dtype=dtype, page=page, sizes=sizes)
        hi = _log_int(rng, 100, 2300)
        return dict(op=op, B=rng.randint(1, 5), new_lo=hi // 3, new_hi=hi, hist=4096, both=False, Hq=Hq, Hkv=Hkv, d=d,
                    rot=rot, layout=layout, affine=rng.random() < 0.5, dtype=dtype, page=page, sizes=sizes)
    if op == "plan":
        tree = rng.random() < 0.6
        return dict(op=op, B=_log_int(rng, 1, 500), tree=tree, new_lo=1, new_hi=_log_int(rng, 1, 64),
                    hist=_log_int(rng, 100, 30000), page=page, pad=rng.choice([0, 0, rng.randint(1, 2000)]), sizes=sizes)
    if op == "commit":
        return dict(op=op, B=_log_int(rng, 1, 48), layers=_log_int(rng, 1, 32), new_lo=8, new_hi=rng.randint(8, 60),
                    most=rng.randint(1, 8), hist=rng.randint(0, 300), Hkv=min(Hkv, 8), d=d,
                    dtype=rng.choice(["bf16", "bf16", "f32"]), page=page, sizes=sizes)
    hi = _log_int(rng, 16, 20000)
    return dict(op=op, B=_log_int(rng, 1, 32), new_lo=1, new_hi=_log_int(rng, 1, 60), hist_lo=hi // 5, hist_hi=hi,
                Hq=Hq, Hkv=Hkv, d=d, window=0 if rng.random() < 0.5 else _log_int(rng, 1, 8192), page=page, sizes=sizes)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_BASE = 500000.0  # rotary base of long-context models
_EPS = 1e-6


def _frequencies(rot):
    i = torch.arange(rot // 2, dtype=torch.float64)
    return _BASE ** (-2.0 * i / rot)


def _gen(seed, dev="cuda"):
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) & 0x7FFFFFFFFFFF)
    return g


def _lens(case):
    """(new tokens, cached tokens before them) of every sequence: the case's sizes."""
    rng = random.Random(case["sizes"])
    B = case["B"]
    new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(B)]
    if "hist_lo" in case:
        return new, [rng.randint(case["hist_lo"], case["hist_hi"]) for _ in range(B)]
    return new, [rng.randint(0, case["hist"]) for _ in range(B)]


def _ends(case):
    """Sequences of a plan that end in this step: one of 16 where there are trees."""
    rng = random.Random(case["sizes"] + 1)
    return [case["tree"] and rng.random() < 1 / 16 for _ in range(case["B"])]


def _tree(rng, n):
    """Parents of a drafted tree, breadth first: a root after the last cached token,
    then each token below one of the few before it in order of probability."""
    wide = rng.choice([2, 3, 4, 8])
    return [-1 if i == 0 else rng.randint(max(0, (i - 1) // wide - 1), max(0, (i - 1) // wide)) for i in range(n)]


def _trees(case, new, seed):
    rng = random.Random(seed * 1000003 + case["sizes"])
    return [_tree(rng, n) for n in new]


def _indptr(new):
    at = [0]
    for n in new:
        at.append(at[-1] + n)
    return at


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _table(g, lens, page, spare=3):
    """Block tables with the sequences' pages scattered over a pool; (table, pages in the pool)."""
    need = [max((n + page - 1) // page, 1) for n in lens]
    total = sum(need) + spare
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    bt = torch.zeros((len(lens), max(need)), dtype=torch.int32, device="cuda")
    o = 0
    for b, n in enumerate(need):
        bt[b, :n] = perm[o:o + n]
        o += n
    return bt, total


def _masks(trees, words):
    """Ancestor masks [tokens, words]: bit j of a row is token j of its own sequence's tree."""
    rows = []
    for t in trees:
        own_rows = []
        for i, p in enumerate(t):
            m = (own_rows[p] if p >= 0 else 0) | 1 << i
            own_rows.append(m)
        rows += own_rows
    flat = [(m >> 32 * w) & 0xFFFFFFFF for m in rows for w in range(words)]
    return torch.tensor(flat, dtype=torch.int64).to(torch.int32).view(-1, words).cuda()


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(op=op, case=case)

    def randn(*shape, dt=torch.float32):
        return torch.randn(shape, generator=g, device="cuda", dtype=dt)

    if op in ("norm_rotate", "norm_backward"):
        n, H, d, dt = case["n"], case["H"], case["d"], _DT[case["dtype"]]
        s.update(x=3.0 * randn(n, H, d, dt=dt), freq=_frequencies(case["rot"]), w=1.0 + 0.2 * randn(d), alpha=None,
                 beta=None)
        if case["affine"]:
            s["alpha"], s["beta"] = 1.0 + 0.1 * randn(H, d), 0.1 * randn(H, d)
        if case["pos"] == "far":  # decoding rows: anywhere in a long context
            s["pos"] = torch.randint(0, 131072, (n,), generator=g, device="cuda", dtype=torch.int32)
        else:                     # tokens of sequences of up to 8192
            s["pos"] = (torch.arange(n, device="cuda") % 8192).to(torch.int32)
        if op == "norm_backward":
            s["dy"] = randn(n, H, d, dt=dt)
    elif op == "norm_append":
        dt, Hq, Hkv, d = _DT[case["dtype"]], case["Hq"], case["Hkv"], case["d"]
        new, hist = _lens(case)
        n = sum(new)
        bt, pages = _table(g, [a + b for a, b in zip(new, hist)], case["page"])
        seq = torch.cat([torch.full((m,), b) for b, m in enumerate(new)]).cuda()
        at = torch.cat([torch.arange(h, h + m) for m, h in zip(new, hist)]).cuda()
        slots = bt[seq, at // case["page"]].long() * case["page"] + at % case["page"]
        pos = at
        if case["both"]:  # trees: a token's position is its depth below the last cached token
            depth = []
            for t in _trees(case, new, seed):
                o = len(depth)
                for p in t:
                    depth.append(0 if p < 0 else depth[o + p] + 1)
            first = torch.cat([torch.full((m,), h) for m, h in zip(new, hist)])
            pos = (first + torch.tensor(depth)).cuda()
        # q, k and v as the projection leaves them: parts of one row a token
        packed = 2.0 * randn(n, Hq + 2 * Hkv, d, dt=dt)
        s.update(q=packed[:, :Hq], k=packed[:, Hq:Hq + Hkv], v=packed[:, Hq + Hkv:],
                 q_out=2.0 * randn(n, Hq, d, dt=dt) if case["both"] else None, slots=slots.to(torch.int32),
                 pos=pos.to(torch.int32), freq=_frequencies(case["rot"]), qw=1.0 + 0.2 * randn(d), kw=1.0 + 0.2 * randn(d),
                 kc=randn(pages, case["page"], Hkv, d, dt=dt), vc=randn(pages, case["page"], Hkv, d, dt=dt), aff=None)
        if case["affine"]:
            s["aff"] = [1.0 + 0.1 * randn(Hq, d), 0.1 * randn(Hq, d), 1.0 + 0.1 * randn(Hq, d), 0.1 * randn(Hq, d)]
    elif op == "plan":
        new, hist = _lens(case)
        page = case["page"]
        ends = _ends(case)
        new = [-1 if e else m for m, e in zip(new, ends)]
        # a sequence holds the pages of its cached tokens; ended ones give theirs back
        held = [(h + page - 1) // page for h in hist]
        width = max((h + max(m, 0) + page - 1) // page for m, h in zip(new, hist)) + 1
        taken, spare = sum(held), sum((max(m, 0) + page - 1) // page + 1 for m in new) + 5
        perm = torch.randperm(taken + spare, generator=g, device="cuda").to(torch.int32)
        row = torch.repeat_interleave(torch.arange(len(held)), torch.tensor(held)).cuda()
        col = torch.cat([torch.arange(h) for h in held]).cuda()
        bt = torch.full((len(new), width), -1, dtype=torch.int32, device="cuda")
        bt[row, col] = perm[:taken]
        free = torch.full((taken + spare,), -1, dtype=torch.int32, device="cuda")
        free[:spare] = perm[taken:]
        live = [max(m, 0) for m in new]
        n = sum(live) + case["pad"]
        parents = None
        if case["tree"]:
            parents = [p for t in _trees(case, live, seed) for p in t]
            parents = _i32(parents + [0] * (n - len(parents)))
        s.update(cache_lens=_i32(hist), new_lens=_i32(new), held=_i32(held), free=free, count=_i32([spare]), bt=bt, n=n,
                 page=page, parents=parents, max_tree=64 if case["tree"] else 0)
        if own:
            import efficient_long_context_gb300 as ola

            B = len(new)
            s["ws"] = torch.empty(256, dtype=torch.uint8, device="cuda")
            s["out"] = ola.orthros_plan_step_buffers(B, n, s["max_tree"])
    elif op == "tree_attend":
        new, hist = _lens(case)
        total = [a + b for a, b in zip(new, hist)]
        trees = _trees(case, new, seed)
        bt, pages = _table(g, total, case["page"])
        kv = (pages, case["page"], case["Hkv"], case["d"])
        words = (max(new) + 31) // 32
        s.update(q=randn(sum(new), case["Hq"], case["d"], dt=torch.bfloat16), kc=randn(*kv, dt=torch.bfloat16),
                 vc=randn(*kv, dt=torch.bfloat16), bt=bt, indptr=_i32(_indptr(new)), kv_lens=_i32(total),
                 mask=_masks(trees, words), new=new, total=total, words=words,
                 window=case["window"] if case["window"] > 0 else max(total))
        if own:
            import efficient_long_context_gb300 as ola

            s["ws"] = torch.empty(ola.orthros_tree_attention_workspace_size(
                case["B"], sum(new), max(new), case["Hq"], case["Hkv"], case["d"], bt.shape[1], case["page"]),
                dtype=torch.uint8, device="cuda")
    else:
        new, hist = _lens(case)
        total = [a + b for a, b in zip(new, hist)]
        bt, pages = _table(g, total, case["page"])
        kv = (case["layers"], pages, case["page"], case["Hkv"], case["d"])
        # The accepted path: the root, then tokens of the tree behind the path's length, so that a
        # pass leaves in place what it reads and can be repeated on the same cache.
        rng = random.Random(seed * 7919 + case["sizes"])
        acc, count = [], []
        for m in new:
            k = rng.randint(1, min(case["most"], m // 2))
            path = [0] + sorted(rng.sample(range(k, m), k - 1))
            acc.append(path + [0] * (case["most"] - k))
            count.append(k)
        s.update(kc=randn(*kv, dt=_DT[case["dtype"]]), vc=randn(*kv, dt=_DT[case["dtype"]]), bt=bt,
                 indptr=_i32(_indptr(new)), kv_lens=_i32(total), acc=_i32(acc), count=_i32(count))
        if own:
            s["ws"] = torch.empty(256, dtype=torch.uint8, device="cuda")
            s["lens"] = torch.empty(case["B"], dtype=torch.int32, device="cuda")
    if "freq" in s:
        if own:
            import efficient_long_context_gb300 as ola

            s["steps"] = ola.orthros_rotary_steps(s["freq"]).cuda()
            if op == "norm_append":
                s["ws"] = torch.empty(256, dtype=torch.uint8, device="cuda")
            if op == "norm_backward":
                s["ws"] = torch.empty(ola.orthros_norm_rotate_backward_workspace_size(
                    case["n"], case["H"], case["d"], s["x"].dtype), dtype=torch.uint8, device="cuda")
        s["freq"] = s["freq"].cuda()
    return s


# ---------------------------------------------------------------------------
# plain forms (32 bits, angles in 64)
# ---------------------------------------------------------------------------
def _pairs(x, rot, layout):
    if layout == "half":
        return x[..., :rot // 2], x[..., rot // 2:rot]
    return x[..., 0:rot:2], x[..., 1:rot:2]


def _join(a, b, rest, layout):
    if layout == "half":
        return torch.cat([a, b, rest], -1)
    return torch.cat([torch.stack([a, b], -1).flatten(-2), rest], -1)


def _turned(y, pos, freq, layout, sign=1.0):
    a = pos.double()[:, None] * freq[None, :]
    c, s = torch.cos(a).float()[:, None, :], (sign * torch.sin(a)).float()[:, None, :]
    a, b = _pairs(y, 2 * freq.numel(), layout)
    return _join(a * c - b * s, a * s + b * c, y[..., 2 * freq.numel():], layout)


def _plain_norm(x, w, pos, freq, layout, alpha=None, beta=None):
    y = x.float()
    y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + _EPS) * w
    if alpha is not None:
        y = y * alpha + beta
    return _turned(y, pos, freq, layout).to(x.dtype)


def _plain_norm_backward(s):
    layout, w, x = s["case"]["layout"], s["w"], s["x"].float()
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + _EPS)
    xh = x * r
    g = _turned(s["dy"].float(), s["pos"], s["freq"], layout, -1.0)
    a = w if s["alpha"] is None else w * s["alpha"]
    u = g * a
    out = {"dx": (r * (u - xh * (u * xh).mean(-1, keepdim=True))).to(s["x"].dtype)}
    S = (g * xh).sum(0)
    if s["alpha"] is None:
        out["d_weight"] = S.sum(0)
    else:
        out.update(d_weight=(S * s["alpha"]).sum(0), d_alpha=S * w, d_beta=g.sum(0))
    return out


def _plain_append(s):
    layout, al = s["case"]["layout"], s["aff"] or [None] * 4
    out = {"q": _plain_norm(s["q"], s["qw"], s["pos"], s["freq"], layout, al[0], al[1])}
    if s["q_out"] is not None:
        out["q_out"] = _plain_norm(s["q_out"], s["qw"], s["pos"], s["freq"], layout, al[2], al[3])
    rows = s["slots"].long()
    s["kc"].flatten(0, 1)[rows] = _plain_norm(s["k"], s["kw"], s["pos"], s["freq"], layout)
    s["vc"].flatten(0, 1)[rows] = s["v"]
    return dict(out, k_cache=s["kc"], v_cache=s["vc"])


def _plain_plan(s):
    """Free pages are a stack: ended sequences push theirs, growing ones then take from
    the top, in the order of the sequences. Rows behind the last token are -1 (position 0)."""
    page, n, dev = s["page"], s["n"], s["bt"].device
    L, m, held = s["cache_lens"].long(), s["new_lens"].long(), s["held"].long()
    ended, live = m < 0, m.clamp(min=0)
    kv = torch.where(ended, 0, L + live)
    ends = torch.cumsum(live, 0)
    indptr = torch.cat([ends.new_zeros(1), ends])
    free, count = s["free"].clone(), s["count"].long()
    back = torch.where(ended, held, 0)
    col = torch.arange(s["bt"].shape[1], device=dev)
    give = col[None, :] < back[:, None]
    at = (count + torch.cumsum(back, 0) - back)[:, None] + col[None, :]
    free[at[give]] = s["bt"][give]
    count = count + back.sum()
    need = torch.where(ended, 0, torch.maximum(held, (kv + page - 1) // page))
    grow = torch.where(ended, 0, need - held)
    off = torch.cumsum(grow, 0) - grow
    bt = s["bt"].clone()
    new = (col[None, :] >= held[:, None]) & (col[None, :] < need[:, None])
    src = count - 1 - (off[:, None] + col[None, :] - held[:, None])
    bt[new] = free[src[new]]
    i = torch.arange(n, device=dev)
    seq = torch.searchsorted(ends, i, right=True)
    real = seq < L.numel()
    sq = seq.clamp(max=L.numel() - 1)
    j = i - indptr[sq]
    t = L[sq] + j
    slot = bt[sq, (t // page).clamp(max=bt.shape[1] - 1)].long() * page + t % page
    pos, mask = t, None
    if s["parents"] is not None:
        words = (s["max_tree"] + 31) // 32
        bits = torch.zeros((n, words), dtype=torch.int64, device=dev)
        at, depth = torch.where(real, j, -1), torch.zeros_like(i)
        for _ in range(s["max_tree"]):
            up = at >= 0
            w = at.clamp(min=0)
            bits.scatter_add_(1, (w // 32)[:, None], torch.where(up, 1 << w % 32, 0)[:, None])
            at = torch.where(up, s["parents"].long()[(indptr[sq] + w).clamp(max=n - 1)], -1)
            depth += at >= 0
        mask = torch.where(bits >= 2 ** 31, bits - 2 ** 32, bits).to(torch.int32)
        pos = L[sq] + depth
    i32 = torch.int32
    out = {"q_indptr": indptr.to(i32), "kv_lens": kv.to(i32), "pages_held": need.to(i32),
           "free_count": (count - grow.sum()).to(i32), "token_seq": torch.where(real, seq, -1).to(i32),
           "token_pos": torch.where(real, pos, 0).to(i32), "token_slots": torch.where(real, slot, -1).to(i32),
           "block_table": bt, "free_pages": free}
    return out if mask is None else dict(out, tree_mask=mask)


def _bits(mask, n):
    """Mask words [rows, words] as truth values [rows, n]."""
    j = torch.arange(n, device=mask.device)
    return (mask[:, j // 32] >> (j % 32) & 1).bool()


def _plain_tree(s):
    q, w, page = s["q"], s["window"], s["kc"].shape[1]
    Hq, d = q.shape[1:]
    Hkv = s["kc"].shape[2]
    o = torch.empty_like(q)
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    i0 = 0
    for b, (n, T) in enumerate(zip(s["new"], s["total"])):
        L = T - n
        seen = _bits(s["mask"][i0:i0 + n], n)
        t = L + seen.sum(-1) - 1  # a token's position: its depth in the tree
        first = max(0, L - w + 1) // page * page
        pages = s["bt"][b, first // page:(T + page - 1) // page].long()
        kk = s["kc"][pages].flatten(0, 1)[:T - first].float()
        vv = s["vc"][pages].flatten(0, 1)[:T - first].float()
        keys = torch.cat([torch.arange(first, L, device=q.device), t])
        hide = keys[None, :] <= t[:, None] - w
        hide[:, L - first:] |= ~seen
        z = torch.einsum("nkgd,jkd->kgnj", q[i0:i0 + n].float().view(n, Hkv, Hq // Hkv, d), kk) * d ** -0.5
        z = z.masked_fill_(hide, float("-inf"))
        m = z.amax(-1, keepdim=True)
        p = torch.exp(z - m)
        l = p.sum(-1, keepdim=True)
        r = torch.einsum("kgnj,jkd->nkgd", p / l, vv)
        o[i0:i0 + n] = r.reshape(n, Hq, d).to(q.dtype)
        lse[i0:i0 + n] = (m + torch.log(l)).squeeze(-1).permute(2, 0, 1).reshape(n, Hq)
        i0 += n
    return {"o": o, "lse": lse}


def _plain_commit(s):
    kc, vc = s["kc"], s["vc"]
    page = kc.shape[2]
    L = s["kv_lens"].long() - (s["indptr"][1:] - s["indptr"][:-1]).long()
    i = torch.arange(s["acc"].shape[1], device=kc.device)
    keep = i[None, :] < s["count"].long()[:, None]
    to = (L[:, None] + i[None, :])[keep]
    fro = (L[:, None] + s["acc"].long())[keep]
    b = torch.arange(L.numel(), device=kc.device)[:, None].expand(keep.shape)[keep]
    to = s["bt"][b, to // page].long() * page + to % page
    fro = s["bt"][b, fro // page].long() * page + fro % page
    for c in (kc, vc):
        c = c.flatten(1, 2)
        c[:, to] = c[:, fro]
    return {"k_cache": kc, "v_cache": vc, "cache_lens": (L + s["count"].long()).to(torch.int32)}


def run(state):
    s = state
    case, op = s["case"], s["op"]
    if own:
        import efficient_long_context_gb300 as ola

        if op == "norm_rotate":
            return ola.orthros_norm_rotate(s["x"], s["pos"], s["steps"], s["w"], _EPS, layout=case["layout"],
                                           alpha=s["alpha"], beta=s["beta"])
        if op == "norm_backward":
            dx, dw, da, db = ola.orthros_norm_rotate_backward(
                s["dy"], s["x"], s["pos"], s["steps"], s["w"], _EPS, layout=case["layout"], alpha=s["alpha"],
                affine_grads=case["affine"], workspace=s["ws"])
            out = {"dx": dx, "d_weight": dw}
            return dict(out, d_alpha=da, d_beta=db) if case["affine"] else out
        if op == "norm_append":
            aff = s["aff"] or [None] * 4
            q, qo = ola.orthros_norm_rotate_append(
                s["q"], s["k"], s["v"], s["kc"], s["vc"], s["slots"], s["pos"], s["steps"], eps=_EPS, q_weight=s["qw"],
                k_weight=s["kw"], layout=case["layout"], q_out=s["q_out"],
                out_positions=s["pos"] if case["both"] else None, alpha_base=aff[0], beta_base=aff[1], alpha_out=aff[2],
                beta_out=aff[3], workspace=s["ws"])
            out = {"q": q, "k_cache": s["kc"], "v_cache": s["vc"]}
            return dict(out, q_out=qo) if case["both"] else out
        if op == "plan":
            p = ola.orthros_plan_step(s["cache_lens"], s["new_lens"], s["held"], s["free"], s["count"], s["bt"], s["page"],
                                      s["n"], parents=s["parents"], max_tree=s["max_tree"], out=s["out"], workspace=s["ws"])
            out = {"q_indptr": p.q_indptr, "kv_lens": p.kv_lens, "pages_held": p.pages_held, "free_count": p.free_count,
                   "token_seq": p.token_seq, "token_pos": p.token_pos, "token_slots": p.token_slots,
                   "block_table": s["bt"], "free_pages": s["free"]}
            return dict(out, tree_mask=p.tree_mask) if case["tree"] else out
        if op == "tree_attend":
            o, lse = ola.orthros_tree_attention(s["q"], s["indptr"], s["kv_lens"], s["mask"], s["kc"], s["vc"], s["bt"],
                                                s["window"], max_new=max(s["new"]), workspace=s["ws"])
            return {"o": o, "lse": lse}
        lens = ola.orthros_tree_commit(s["kc"], s["vc"], s["bt"], s["indptr"], s["kv_lens"], s["acc"], s["count"],
                                       out=s["lens"], workspace=s["ws"])
        return {"k_cache": s["kc"], "v_cache": s["vc"], "cache_lens": lens}
    if op == "norm_rotate":
        return _plain_norm(s["x"], s["w"], s["pos"], s["freq"], case["layout"], s["alpha"], s["beta"])
    return {"norm_backward": _plain_norm_backward, "norm_append": _plain_append, "plan": _plain_plan,
            "tree_attend": _plain_tree, "commit": _plain_commit}[op](s)


# ---------------------------------------------------------------------------
# the work a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op in ("norm_rotate", "norm_backward"):
        e = 2 if case["dtype"] == "bf16" else 4
        n, H, d = case["n"], case["H"], case["d"]
        nel = n * H * d
        aff = 2 * H * d * 4 if case["affine"] else 0
        turn = 3 * n * H * case["rot"]
        if op == "norm_rotate":
            return {"bytes": 2 * nel * e + 4 * n + 4 * d + aff, "flops": turn + (6 if aff else 4) * nel}
        return {"bytes": 3 * nel * e + 4 * n + 8 * d + 3 * aff // 2, "flops": turn + 12 * nel}
    new, hist = _lens(case)
    if op == "norm_append":
        e = 2 if case["dtype"] == "bf16" else 4
        n, Hq, Hkv, d = sum(new), case["Hq"], case["Hkv"], case["d"]
        rows = n * (Hq * (2 if case["both"] else 1) + 2 * Hkv)
        return {"bytes": 2 * rows * d * e + 8 * n + 8 * d + (4 * Hq * d * 4 if case["affine"] else 0),
                "flops": (rows - n * Hkv) * (3 * case["rot"] + 4 * d)}
    if op == "plan":
        live = [0 if e else m for m, e in zip(new, _ends(case))]
        n, B, page = sum(live) + case["pad"], case["B"], case["page"]
        words = 2 if case["tree"] else 0
        grown = sum((h + m + page - 1) // page - (h + page - 1) // page for m, h in zip(live, hist))
        back = sum((h + page - 1) // page for h, e in zip(hist, _ends(case)) if e)
        return {"bytes": 4 * (3 * B + 3 * B + 1 + 2) + 12 * n + 4 * words * n + (4 * n if words else 0) +
                8 * (grown + back), "flops": 0}
    if op == "commit":
        # the expected path: half of the longest, its root already in place
        e = 2 if case["dtype"] == "bf16" else 4
        rows = case["B"] * max(case["most"] - 1, 1) / 2
        return {"bytes": int(case["layers"] * rows * case["Hkv"] * case["d"] * e * 4) + 4 * case["B"] * (case["most"] + 4),
                "flops": 0}
    w, d, Hq = case["window"], case["d"], case["Hq"]
    pairs, keys = 0, 0
    for m, h in zip(new, hist):
        seen = h if w == 0 else min(h, w - 1)
        pairs += m * seen + m  # the cached keys and the token itself; its few ancestors are left out
        keys += seen + m
    n = sum(new)
    return {"bytes": 2 * n * Hq * d * 2 + 4 * n * Hq + 2 * keys * case["Hkv"] * d * 2, "flops": 4 * d * Hq * pairs}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _exact_rotation(x, pos, freq, layout, sign):
    """Rows of complex numbers times e^(i sign t freq)."""
    r = 2 * freq.numel()
    if layout == "half":
        re, im = list(range(r // 2)), list(range(r // 2, r))
    else:
        re, im = list(range(0, r, 2)), list(range(1, r, 2))
    z = torch.complex(x[..., re], x[..., im])
    th = sign * torch.outer(pos.to(torch.float64), freq.to(x.device))
    z = z * torch.polar(torch.ones_like(th), th).unsqueeze(1)
    y = x.clone()
    y[..., re] = z.real
    y[..., im] = z.imag
    return y


def _exact_norm(x, w, alpha, beta):
    x = x.double()
    z = x * torch.rsqrt(torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / x.shape[-1] + _EPS) * w.double()
    return z if alpha is None else z * alpha.double() + beta.double()


def _exact_backward(s, layout):
    """The gradient through the 64-bit definition, by the chain rule of x |-> x (x.x/d + eps)^(-1/2)."""
    x = s["x"].double()
    d = x.shape[-1]
    v = (x * x).sum(-1, keepdim=True) / d + _EPS
    g = _exact_rotation(s["dy"].double(), s["pos"], s["freq"], layout, -1.0)
    w = s["w"].double()
    gain = w.expand(x.shape[1:]) if s["alpha"] is None else w * s["alpha"].double()
    gz = g * gain
    dx = gz * v ** -0.5 - x * v ** -1.5 * (gz * x).sum(-1, keepdim=True) / d
    per_head = torch.einsum("nhd,nhd->hd", g, x * v ** -0.5)
    if s["alpha"] is None:
        return {"dx": dx, "d_weight": per_head.sum(0)}
    return {"dx": dx, "d_weight": torch.einsum("hd,hd->d", per_head, s["alpha"].double()), "d_alpha": per_head * w,
            "d_beta": torch.einsum("nhd->hd", g)}


def _exact_tree(s, case):
    q, page, w = s["q"].double(), case["page"], s["window"]
    d, Hq, Hkv = q.shape[-1], case["Hq"], case["Hkv"]
    o, lse = torch.empty_like(q), torch.empty(q.shape[:2], dtype=torch.float64, device=q.device)
    bits = s["mask"].cpu().tolist()
    start = 0
    for b, (n, T) in enumerate(zip(s["new"], s["total"])):
        L = T - n
        seen = torch.zeros((n, T), dtype=torch.bool)
        at = []
        for i in range(n):
            row = sum((x % 2 ** 32) << 32 * k for k, x in enumerate(bits[start + i]))
            at.append(L + bin(row).count("1") - 1)
            seen[i, max(0, at[i] - w + 1):L] = True
            for j in range(n):
                seen[i, L + j] = bool(row >> j & 1)
        for i in range(n):
            for j in range(n):
                if at[j] <= at[i] - w:
                    seen[i, L + j] = False
        seen = seen.to(q.device)
        idx = torch.arange(T, device=q.device)
        pg = s["bt"][b].long()[torch.div(idx, page, rounding_mode="floor")]
        for h in range(Hkv):
            kh, vh = s["kc"][pg, idx % page, h].double(), s["vc"][pg, idx % page, h].double()
            for j in range(h * (Hq // Hkv), (h + 1) * (Hq // Hkv)):
                z = (q[start:start + n, j] @ kh.T) / math.sqrt(d)
                z = torch.where(seen, z, torch.full_like(z, -math.inf))
                e = torch.logsumexp(z, -1)
                o[start:start + n, j] = torch.exp(z - e.unsqueeze(1)) @ vh
                lse[start:start + n, j] = e
        start += n
    return {"o": o, "lse": lse}


def exact(case, seed):
    op, layout = case["op"], case.get("layout")
    if op == "plan":
        return None  # whole numbers only
    s = prepare(case, seed)
    if op == "norm_rotate":
        return _exact_rotation(_exact_norm(s["x"], s["w"], s["alpha"], s["beta"]), s["pos"], s["freq"], layout, 1.0)
    if op == "norm_backward":
        return _exact_backward(s, layout)
    if op == "norm_append":
        aff = s["aff"] or [None] * 4
        out = {"q": _exact_rotation(_exact_norm(s["q"], s["qw"], aff[0], aff[1]), s["pos"], s["freq"], layout, 1.0)}
        if case["both"]:
            out["q_out"] = _exact_rotation(_exact_norm(s["q_out"], s["qw"], aff[2], aff[3]), s["pos"], s["freq"], layout, 1.0)
        kc, vc, page = s["kc"].double(), s["vc"].double(), case["page"]
        pg, at = torch.div(s["slots"].long(), page, rounding_mode="floor"), s["slots"].long() % page
        kc[pg, at] = _exact_rotation(_exact_norm(s["k"], s["kw"], None, None), s["pos"], s["freq"], layout, 1.0)
        vc[pg, at] = s["v"].double()
        return dict(out, k_cache=kc, v_cache=vc)
    if op == "tree_attend":
        return _exact_tree(s, case) if work(case)["flops"] < 4e12 else None
    if case["layers"] > 8:
        return None  # rows moved, nothing computed; the smaller case stands for it
    new, hist = _lens(case)
    kc, vc = s["kc"].double(), s["vc"].double()
    bt, acc, count, page = s["bt"].tolist(), s["acc"].tolist(), s["count"].tolist(), case["page"]
    for b, L in enumerate(hist):
        for i in range(count[b]):  # in order: a token never moves behind one that is still to move
            fro, to = L + acc[b][i], L + i
            for c in (kc, vc):
                c[:, bt[b][to // page], to % page] = c[:, bt[b][fro // page], fro % page]
    return {"k_cache": kc, "v_cache": vc, "cache_lens": None}
