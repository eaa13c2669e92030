"""Rotary positions, the paged append that applies them, and the attention of
new tokens over the paged cache: the calls, their plain forms and their exact
values.

Four operators that a layer runs in this order when its tokens carry rotary
positions:

rotate           y = m R(t) (alpha (.) x + beta): the per-(head, channel) affine
                 of a query stream, then the rotation of pair i by the angle
                 t * freq[i], in the half layout (channels i, i + r/2) or the
                 interleaved one (2i, 2i + 1) of the first r channels.
rotate_backward  dx, d_alpha, d_beta of the same.
append           new keys rotated and written with their values into the pages
                 of a paged cache; both query streams rotated in the same call.
attend           new tokens of a batch of sequences (ragged: one token each, a
                 chunk, or both mixed) over the paged cache that already holds
                 their keys: token at position t sees keys max(0, t-w+1) .. t.

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
        # both queries of 32 decoding pairs at 16K-32K positions: launch latency counts
        dict(name="rotate_decode_64", op="rotate", n=64, H=32, d=128, rot=128, layout="half", affine=True,
             dtype="bf16", pos="far"),
        # the queries of a fine-tuning step, 4 x 8192 tokens
        dict(name="rotate_sft_32768", op="rotate", n=32768, H=32, d=128, rot=128, layout="interleaved",
             affine=True, dtype="bf16", pos="seq"),
        # keys of an odd number of tokens, a quarter of the head rotated, fp32
        dict(name="rotate_keys_f32_4099", op="rotate", n=4099, H=4, d=64, rot=16, layout="half", affine=False,
             dtype="f32", pos="seq"),
        # gradient of the fine-tuning queries, with the affine's
        dict(name="rotate_grad_sft_32768", op="rotate_backward", n=32768, H=32, d=128, rot=128, layout="half",
             affine=True, dtype="bf16", pos="seq"),
        # gradient of a small fp32 model's queries, odd length, half of the head rotated
        dict(name="rotate_grad_f32_2049", op="rotate_backward", n=2049, H=4, d=64, rot=32, layout="interleaved",
             affine=True, dtype="f32", pos="seq"),
        # 32 sequences decode one token pair each
        dict(name="append_decode_32", op="append", B=32, lens="decode", new=1, cap=2048, Hq=32, Hkv=8, d=128,
             rot=128, layout="half", affine=False, dtype="bf16", page=64, sizes=11),
        # prompts of five sequences, 8191 tokens in all, small pages
        dict(name="append_chunks_8191", op="append", B=5, lens="ragged", new=8191, cap=4096, Hq=32, Hkv=8, d=128,
             rot=128, layout="interleaved", affine=True, dtype="bf16", page=16, sizes=12),
        # one user, one token, 32K of history: latency and the split of the key axis
        dict(name="attend_one_32k", op="attend", B=1, new_lo=1, new_hi=1, hist_lo=32767, hist_hi=32767, Hq=32, Hkv=8,
             d=128, window=0, page=64, sizes=11),
        # 32 sequences decode over 16K-32K of history
        dict(name="attend_decode_32", op="attend", B=32, new_lo=1, new_hi=1, hist_lo=16384, hist_hi=32768, Hq=32,
             Hkv=8, d=128, window=0, page=64, sizes=11),
        # a serving step: some sequences decode, some append up to 64 tokens; windowed stream, small pages
        dict(name="attend_mixed_24", op="attend", B=24, new_lo=1, new_hi=64, hist_lo=1000, hist_hi=20000, Hq=32,
             Hkv=8, d=128, window=4096, page=16, sizes=12),
        # a prompt's chunk of 2048 tokens behind 30000 cached ones, window 4096
        dict(name="attend_chunk_2048", op="attend", B=1, new_lo=2048, new_hi=2048, hist_lo=30000, hist_hi=30000, Hq=32,
             Hkv=8, d=128, window=4096, page=64, sizes=11),
        # two long chunks over all of 16K-24K tokens of history
        dict(name="attend_full_2x4000", op="attend", B=2, new_lo=3700, new_hi=4200, hist_lo=16384, hist_hi=24576,
             Hq=32, Hkv=8, d=128, window=0, page=64, sizes=11),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "rotate_backward", "append", "attend", "attend"])
    d = rng.choice([64, 128, 128])
    Hq, Hkv = rng.choice([(32, 8), (32, 8), (16, 16), (4, 4), (8, 2), (12, 4)])
    layout = rng.choice(["half", "interleaved"])
    rot = rng.choice([r for r in (16, 32, 48, 64, 96, 128) if r <= d])
    if op in ("rotate", "rotate_backward"):
        return dict(op=op, n=_log_int(rng, 1, 32768), H=rng.choice([Hq, Hkv]), d=d, rot=rot, layout=layout,
                    affine=rng.random() < 0.6 or op == "rotate_backward", dtype=rng.choice(["bf16", "bf16", "f32"]),
                    pos=rng.choice(["seq", "far"]))
    page = rng.choice([8, 16, 32, 48, 64, 128])
    if op == "append":
        if rng.random() < 0.5:
            return dict(op=op, B=_log_int(rng, 1, 64), lens="decode", new=1, cap=2048, Hq=Hq, Hkv=Hkv, d=d, rot=rot,
                        layout=layout, affine=rng.random() < 0.5, dtype=rng.choice(["bf16", "bf16", "f32"]),
                        page=page, sizes=rng.randint(0, 9999))
        return dict(op=op, B=rng.randint(1, 9), lens="ragged", new=_log_int(rng, 1, 8192), cap=4096, Hq=Hq, Hkv=Hkv,
                    d=d, rot=rot, layout=layout, affine=rng.random() < 0.5, dtype=rng.choice(["bf16", "bf16", "f32"]),
                    page=page, sizes=rng.randint(0, 9999))
    window = 0 if rng.random() < 0.4 else _log_int(rng, 1, 8192)
    kind = rng.random()
    if kind < 0.35:    # decoding
        B, new = _log_int(rng, 1, 32), (1, 1)
        hist = (0, _log_int(rng, 16, 32768))
    elif kind < 0.7:   # mixed
        B, new = _log_int(rng, 1, 24), (1, _log_int(rng, 2, 128))
        hist = (0, _log_int(rng, 16, 20000))
    else:              # chunks
        B = rng.randint(1, 2)
        n = _log_int(rng, 100, 4000)
        new = (n, n + 200)
        hist = (0, _log_int(rng, 16, 24000))
    return dict(op="attend", B=B, new_lo=new[0], new_hi=new[1], hist_lo=hist[0], hist_hi=hist[1], Hq=Hq, Hkv=Hkv, d=d,
                window=window, page=page, sizes=rng.randint(0, 9999))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_BASE = 500000.0  # rotary base of long-context models


def _frequencies(rot):
    """Long-context frequencies: long wavelengths (past 8192 positions)
    stretched eightfold, short ones (below 2048) kept, a linear blend between."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = _BASE ** (-2.0 * i / rot)
    turns = 8192.0 * f / (2.0 * math.pi)
    s = ((turns - 1.0) / 3.0).clamp(0.0, 1.0)
    return (1.0 - s) * f / 8.0 + s * f


def _gen(seed, dev="cuda"):
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) & 0x7FFFFFFFFFFF)
    return g


def _steps(freq):
    import efficient_long_context_gb300 as ola

    return ola.orthros_rotary_steps(freq).cuda()


def _lens(case):
    """(new tokens, cached tokens before them) of every sequence: the case's sizes."""
    rng = random.Random(case["sizes"])
    B = case["B"]
    if case["op"] == "append":
        if case["lens"] == "decode":
            return [1] * B, [rng.randint(0, case["cap"] - 1) for _ in range(B)]
        cuts = sorted(rng.randint(0, case["new"]) for _ in range(B - 1))
        ends = cuts + [case["new"]]
        new = [b - a for a, b in zip([0] + cuts, ends)]
        return new, [rng.randint(0, case["cap"]) for _ in range(B)]
    lo, hi, h0, h1 = case["new_lo"], case["new_hi"], case["hist_lo"], case["hist_hi"]
    if hi > lo and hi <= 128:  # a serving step: two of three sequences decode
        new = [1 if rng.random() < 0.66 else rng.randint(lo, hi) for _ in range(B)]
    else:
        new = [rng.randint(lo, hi) for _ in range(B)]
    return new, [rng.randint(h0, h1) for _ in range(B)]


def _pages(g, lens, page, Hkv, d, dt):
    """A page pool with the sequences' pages scattered over it."""
    need = [max((n + page - 1) // page, 1) for n in lens]
    mp = max(need)
    total = sum(need) + 3
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    bt = torch.zeros((len(lens), mp), dtype=torch.int32, device="cuda")
    o = 0
    for b, n in enumerate(need):
        bt[b, :n] = perm[o:o + n]
        o += n
    kc = torch.randn((total, page, Hkv, d), generator=g, device="cuda", dtype=dt)
    vc = torch.randn((total, page, Hkv, d), generator=g, device="cuda", dtype=dt)
    return kc, vc, bt


def prepare(case, seed):
    g = _gen(seed)
    op, d = case["op"], case["d"]

    def randn(*shape, dt=torch.float32):
        return torch.randn(shape, generator=g, device="cuda", dtype=dt)

    if op in ("rotate", "rotate_backward"):
        n, H, dt = case["n"], case["H"], _DT[case["dtype"]]
        s = dict(op=op, case=case, x=randn(n, H, d, dt=dt), freq=_frequencies(case["rot"]), alpha=None, beta=None)
        if case["affine"]:
            s["alpha"] = 1.0 + 0.1 * randn(H, d)
            s["beta"] = 0.1 * randn(H, d)
        if case["pos"] == "far":  # decoding rows: anywhere in a long context
            s["pos"] = torch.randint(0, 131072, (n,), generator=g, device="cuda", dtype=torch.int32)
        else:                     # tokens of sequences of up to 8192
            s["pos"] = (torch.arange(n, device="cuda") % 8192).to(torch.int32)
        if op == "rotate_backward":
            s["dy"] = randn(n, H, d, dt=dt)
    elif op == "append":
        dt, Hq, Hkv = _DT[case["dtype"]], case["Hq"], case["Hkv"]
        new, hist = _lens(case)
        kc, vc, bt = _pages(g, [a + b for a, b in zip(new, hist)], case["page"], Hkv, d, dt)
        seq = torch.cat([torch.full((n,), b, dtype=torch.int32) for b, n in enumerate(new)])
        pos = torch.cat([torch.arange(h, h + n, dtype=torch.int32) for n, h in zip(new, hist)])
        n = int(seq.numel())
        # the output stream: every sequence's last new token
        outp = torch.tensor([h + m - 1 for m, h in zip(new, hist) if m > 0], dtype=torch.int32)
        s = dict(op=op, case=case, q=randn(n, Hq, d, dt=dt), k=randn(n, Hkv, d, dt=dt), v=randn(n, Hkv, d, dt=dt),
                 q_out=randn(int(outp.numel()), Hq, d, dt=dt), out_pos=outp.cuda(), seq=seq.cuda(), pos=pos.cuda(),
                 kc=kc, vc=vc, bt=bt, freq=_frequencies(case["rot"]), aff=None)
        if case["affine"]:
            s["aff"] = [1.0 + 0.1 * randn(Hq, d), 0.1 * randn(Hq, d), 1.0 + 0.1 * randn(Hq, d), 0.1 * randn(Hq, d)]
    else:
        new, hist = _lens(case)
        total = [a + b for a, b in zip(new, hist)]
        kc, vc, bt = _pages(g, total, case["page"], case["Hkv"], d, torch.bfloat16)
        indptr = [0]
        for m in new:
            indptr.append(indptr[-1] + m)
        s = dict(op=op, case=case, q=randn(indptr[-1], case["Hq"], d, dt=torch.bfloat16), kc=kc, vc=vc, bt=bt,
                 indptr=torch.tensor(indptr, dtype=torch.int32).cuda(),
                 kv_lens=torch.tensor(total, dtype=torch.int32).cuda(), new=new, total=total,
                 window=case["window"] if case["window"] > 0 else max(total))
    if own:
        import efficient_long_context_gb300 as ola

        if op == "attend":
            c = case
            s["ws"] = torch.empty(ola.orthros_chunk_attention_workspace_size(
                c["B"], s["q"].shape[0], max(s["new"]), c["Hq"], c["Hkv"], c["d"], s["bt"].shape[1], c["page"]),
                dtype=torch.uint8, device="cuda")
        else:
            s["steps"] = _steps(s["freq"])
        if op == "append":
            s["ws"] = torch.empty(256, dtype=torch.uint8, device="cuda")
        if op == "rotate_backward":
            s["ws"] = torch.empty(ola.orthros_rotate_backward_workspace_size(case["n"], case["H"], d, s["x"].dtype),
                                  dtype=torch.uint8, device="cuda")
    else:
        s["freq"] = s["freq"].cuda() if "freq" in s else None
    return s


# ---------------------------------------------------------------------------
# plain forms (32 bits, angles in 64)
# ---------------------------------------------------------------------------
def _angles(pos, freq):
    a = pos.double()[:, None] * freq[None, :]
    return torch.cos(a).float()[:, None, :], torch.sin(a).float()[:, None, :]


def _pairs(x, rot, layout):
    if layout == "half":
        return x[..., :rot // 2], x[..., rot // 2:rot]
    return x[..., 0:rot:2], x[..., 1:rot:2]


def _join(a, b, rest, layout):
    if layout == "half":
        return torch.cat([a, b, rest], -1)
    return torch.cat([torch.stack([a, b], -1).flatten(-2), rest], -1)


def _plain_rotate(x, pos, freq, layout, alpha=None, beta=None):
    rot = 2 * freq.numel()
    y = x.float()
    if alpha is not None:
        y = y * alpha + beta
    c, s = _angles(pos, freq)
    a, b = _pairs(y, rot, layout)
    return _join(a * c - b * s, a * s + b * c, y[..., rot:], layout).to(x.dtype)


def _plain_rotate_backward(dy, x, pos, freq, layout, alpha):
    rot = 2 * freq.numel()
    g = dy.float()
    c, s = _angles(pos, freq)
    a, b = _pairs(g, rot, layout)
    g = _join(a * c + b * s, b * c - a * s, g[..., rot:], layout)
    return (g * alpha).to(x.dtype), (g * x.float()).sum(0), g.sum(0)


def _plain_append(s):
    case = s["case"]
    al = s["aff"] or [None] * 4
    q = _plain_rotate(s["q"], s["pos"], s["freq"], case["layout"], al[0], al[1])
    qo = _plain_rotate(s["q_out"], s["out_pos"], s["freq"], case["layout"], al[2], al[3])
    k = _plain_rotate(s["k"], s["pos"], s["freq"], case["layout"])
    page = s["kc"].shape[1]
    pos = s["pos"].long()
    rows = s["bt"][s["seq"].long(), pos // page].long() * page + pos % page
    s["kc"].flatten(0, 1)[rows] = k
    s["vc"].flatten(0, 1)[rows] = s["v"]
    return {"q": q, "q_out": qo, "k_cache": s["kc"], "v_cache": s["vc"]}


def _plain_attend(s):
    q, d = s["q"], s["q"].shape[-1]
    Hq, Hkv = q.shape[1], s["kc"].shape[2]
    g, page, w, scale = Hq // Hkv, s["kc"].shape[1], s["window"], d ** -0.5
    o = torch.empty_like(q)
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    i0 = 0
    for b, (n, L) in enumerate(zip(s["new"], s["total"])):
        if n == 0:
            continue
        first = max(0, L - n - w + 1) // page * page  # first position any token of the sequence sees, by page
        pages = s["bt"][b, first // page:(L + page - 1) // page].long()
        kk = s["kc"][pages].flatten(0, 1)[:L - first].float()  # [keys, Hkv, d]
        vv = s["vc"][pages].flatten(0, 1)[:L - first].float()
        keys = torch.arange(first, L, device=q.device)
        for r0 in range(0, n, 1024):  # rows in pieces, so that the logits fit
            r1 = min(n, r0 + 1024)
            t = torch.arange(L - n + r0, L - n + r1, device=q.device)
            hide = (keys[None, :] > t[:, None]) | (keys[None, :] < t[:, None] - w + 1)
            qq = q[i0 + r0:i0 + r1].float().view(r1 - r0, Hkv, g, d)
            z = torch.einsum("nkgd,jkd->kgnj", qq, kk) * scale
            z = z.masked_fill_(hide, float("-inf"))
            m = z.amax(-1, keepdim=True)
            p = torch.exp(z - m)
            l = p.sum(-1, keepdim=True)
            r = torch.einsum("kgnj,jkd->nkgd", p / l, vv)
            o[i0 + r0:i0 + r1] = r.reshape(r1 - r0, Hq, d).to(q.dtype)
            lse[i0 + r0:i0 + r1] = (m + torch.log(l)).squeeze(-1).permute(2, 0, 1).reshape(r1 - r0, Hq)
        i0 += n
    return {"o": o, "lse": lse}


def run(state):
    s = state
    case, op = s["case"], s["op"]
    if own:
        import efficient_long_context_gb300 as ola

        if op == "rotate":
            return ola.orthros_rotate(s["x"], s["pos"], s["steps"], layout=case["layout"], alpha=s["alpha"],
                                      beta=s["beta"])
        if op == "rotate_backward":
            dx, da, db = ola.orthros_rotate_backward(s["dy"], s["x"], s["pos"], s["steps"], layout=case["layout"],
                                                     alpha=s["alpha"], workspace=s["ws"])
            return {"dx": dx, "d_alpha": da, "d_beta": db}
        if op == "append":
            aff = s["aff"] or [None] * 4
            q, qo = ola.orthros_rotate_append(
                s["q"], s["k"], s["v"], s["kc"], s["vc"], s["bt"], s["seq"], s["pos"], s["steps"],
                layout=case["layout"], q_out=s["q_out"], out_positions=s["out_pos"], alpha_base=aff[0],
                beta_base=aff[1], alpha_out=aff[2], beta_out=aff[3], workspace=s["ws"])
            return {"q": q, "q_out": qo, "k_cache": s["kc"], "v_cache": s["vc"]}
        o, lse = ola.orthros_chunk_attention(s["q"], s["indptr"], s["kv_lens"], s["kc"], s["vc"], s["bt"],
        s["window"],
                                             max_new=max(s["new"]), workspace=s["ws"])
        return {"o": o, "lse": lse}
    if op == "rotate":
        return _plain_rotate(s["x"], s["pos"], s["freq"], case["layout"], s["alpha"], s["beta"])
    if op == "rotate_backward":
        dx, da, db = _plain_rotate_backward(s["dy"], s["x"], s["pos"], s["freq"], case["layout"], s["alpha"])
        return {"dx": dx, "d_alpha": da, "d_beta": db}
    if op == "append":
        return _plain_append(s)
    return _plain_attend(s)


# ---------------------------------------------------------------------------
# the work a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op, d = case["op"], case["d"]
    if op in ("rotate", "rotate_backward"):
        e = 2 if case["dtype"] == "bf16" else 4
        n, H = case["n"], case["H"]
        nel = n * H * d
        aff = 2 * H * d * 4 if case["affine"] else 0
        if op == "rotate":
            return {"bytes": 2 * nel * e + 4 * n + aff, "flops": 3 * n * H * case["rot"] + (2 * nel if aff else 0)}
        return {"bytes": 3 * nel * e + 4 * n + 3 * H * d * 4, "flops": 3 * n * H * case["rot"] + 4 * nel}
    new, hist = _lens(case)
    if op == "append":
        e = 2 if case["dtype"] == "bf16" else 4
        n, Hq, Hkv = sum(new), case["Hq"], case["Hkv"]
        n_out = sum(1 for m in new if m > 0)
        rows = (n + n_out) * Hq + 2 * n * Hkv
        return {"bytes": 2 * rows * d * e + 12 * n + 4 * n_out + (4 * Hq * d * 4 if case["affine"] else 0),
                "flops": 3 * ((n + n_out) * Hq + n * Hkv) * case["rot"]}
    pairs, keys = 0, 0
    for m, h in zip(new, hist):
        w = case["window"] if case["window"] > 0 else m + h
        # token i of the sequence sees min(w, h + i + 1) keys
        full = max(0, min(m, w - h))  # tokens whose window reaches back to position 0
        pairs += full * h + full * (full + 1) // 2 + (m - full) * w
        keys += m + h - max(0, h - w + 1) if m else 0
    n = sum(new)
    return {"bytes": 2 * n * case["Hq"] * d * 2 + 4 * n * case["Hq"] + 2 * keys * case["Hkv"] * d * 2,
            "flops": 4 * d * case["Hq"] * pairs}


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


def _exact_affine(x, alpha, beta):
    return x.double() if alpha is None else x.double() * alpha.double() + beta.double()


def exact(case, seed):
    s = prepare(case, seed)
    op, layout = case["op"], case.get("layout")
    if op == "rotate":
        return _exact_rotation(_exact_affine(s["x"], s["alpha"], s["beta"]), s["pos"], s["freq"], layout, 1.0)
    if op == "rotate_backward":
        g = _exact_rotation(s["dy"].double(), s["pos"], s["freq"], layout, -1.0)
        return {"dx": g * s["alpha"].double(), "d_alpha": (g * s["x"].double()).sum(0), "d_beta": g.sum(0)}
    if op == "append":
        aff = s["aff"] or [None] * 4
        q = _exact_rotation(_exact_affine(s["q"], aff[0], aff[1]), s["pos"], s["freq"], layout, 1.0)
        qo = _exact_rotation(_exact_affine(s["q_out"], aff[2], aff[3]), s["out_pos"], s["freq"], layout, 1.0)
        k = _exact_rotation(s["k"].double(), s["pos"], s["freq"], layout, 1.0)
        kc, vc = s["kc"].double(), s["vc"].double()
        page = kc.shape[1]
        pos = s["pos"].long()
        pg = s["bt"][s["seq"].long(), torch.div(pos, page, rounding_mode="floor")].long()
        kc[pg, pos % page] = k
        vc[pg, pos % page] = s["v"].double()
        return {"q": q, "q_out": qo, "k_cache": kc, "v_cache": vc}
    if work(case)["flops"] > 6e12:
        return None
    q, page, w = s["q"].double(), s["kc"].shape[1], s["window"]
    d, Hq, Hkv = q.shape[-1], q.shape[1], s["kc"].shape[2]
    o, lse = torch.empty_like(q), torch.empty(q.shape[:2], dtype=torch.float64, device=q.device)
    start = 0
    for b in range(case["B"]):
        n, L = s["new"][b], s["total"][b]
        idx = torch.arange(L, device=q.device)
        pg = s["bt"][b].long()[torch.div(idx, page, rounding_mode="floor")]
        for h in range(Hkv):
            kh = s["kc"][pg, idx % page, h].double()
            vh = s["vc"][pg, idx % page, h].double()
            for a in range(0, n, 512):
                c = min(n, a + 512)
                t = torch.arange(L - n + a, L - n + c, device=q.device).unsqueeze(1)
                lo, hi = max(0, L - n + a - w + 1), L - n + c  # keys any of these rows sees
                seen = (idx[lo:hi] <= t) & (idx[lo:hi] > t - w)
                for j in range(h * (Hq // Hkv), (h + 1) * (Hq // Hkv)):
                    z = (q[start + a:start + c, j] @ kh[lo:hi].T) / math.sqrt(d)
                    z = torch.where(seen, z, torch.full_like(z, -math.inf))
                    e = torch.logsumexp(z, -1)
                    o[start + a:start + c, j] = torch.exp(z - e.unsqueeze(1)) @ vh[lo:hi]
                    lse[start + a:start + c, j] = e
        start += n
    return {"o": o, "lse": lse}
