"""The operators of a loop that decodes several continuations of one prompt (beam
search, parallel samples, a system prompt shared by many users) over the 16-bit paged
cache: new tokens' queries and keys normed and rotated and their keys and values put
into pages, full attention of one token per row over pages that neighbouring rows share,
the choice of the best continuations, and the block table's rows put in their new order.

`run` computes each operator in plain torch operations (32 bits; 64 for angles and for
the scores whose order decides what is kept), or, where `own` is true, by the calls of
this repository's package.

A page holds 128 tokens of every KV head, keys and values bf16 [num_pages, Hkv, 128, 128];
block_table[b, c] is the page of tokens 128 c .. 128 c + 127 of row b, cache_lens[b] the
row's tokens, the new ones included.
"""
import math
import random

import numpy as np
import torch

own = False

BLOCK, D = 128, 128
BASE, EPS = 1.0e7, 1.0e-6


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # four samples of one short prompt: latency
        dict(name="attend-b4-short", op="attend", G=16, Hkv=4, sys=0, groups=1, width=4, lo=1500,
             hi=1500, tail=40, empty=0),
        # a batch of users behind one long system prompt, each with a conversation of its own
        dict(name="attend-b64-system", op="attend", G=16, Hkv=4, sys=16384, groups=64, width=1, lo=100,
             hi=4000, tail=0, empty=0),
        # beam search: 8 prompts with 8 beams each, a few hundred tokens in
        dict(name="attend-8x8-beams", op="attend", G=16, Hkv=4, sys=0, groups=8, width=8, lo=8192,
             hi=32768, tail=300, empty=0),
        # the batch of the decode benchmark, nothing shared
        dict(name="attend-b64-apart", op="attend", G=16, Hkv=4, sys=0, groups=64, width=1, lo=8192,
             hi=32768, tail=0, empty=0),
        # a system prompt, behind it 7 prompts with 5 samples each; 6 query heads per KV head,
        # every fourth row is padding
        dict(name="attend-tree-g6", op="attend", G=6, Hkv=2, sys=3333, groups=7, width=5, lo=1, hi=5000,
             tail=700, empty=4),
        # the second step of one prompt's search
        dict(name="select-1x4", op="select", N=1, W=4, V=32000, K=4, bits=32, pad=0, masked=0.0,
             ended=0.0),
        # 32 prompts with 8 beams, twice the beams kept so that ended ones can be set aside
        dict(name="select-32x8", op="select", N=32, W=8, V=131072, K=16, bits=16, pad=0, masked=0.0,
             ended=0.0),
        # constrained search: most of an odd vocabulary masked, rows padded, ended beams among
        # the live ones
        dict(name="select-19x5-masked", op="select", N=19, W=5, V=50001, K=5, bits=32, pad=47,
             masked=0.9, ended=0.2),
        # the beams of 8 prompts with 32k tokens take their parents' places
        dict(name="reorder-64", op="reorder", B=64, width=8, per_row=256, pages=17000),
        # many rows with long tables, some dropped
        dict(name="reorder-1000", op="reorder", B=1000, width=4, per_row=1024, pages=600000),
        # the new token of 64 rows (the full-attention layers: no index)
        dict(name="append-b64", op="append", S=64, lo=1, hi=1, before=20000, G=16, Hkv=4, R=64,
             layout="half", scaling="yarn", norm=True, index=False),
        # chunks of 8 prompts into the pages of the sparse layers, positions inside a page
        dict(name="append-chunk-16k", op="append", S=8, lo=512, hi=4096, before=777, G=16, Hkv=4, R=64,
             layout="half", scaling="none", norm=True, index=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "select", "select", "reorder", "append"])
    if op == "attend":
        groups, width = rng.choice([(_log(rng, 1, 64), 1), (_log(rng, 1, 8), _log(rng, 1, 8)),
                                    (1, _log(rng, 2, 64))])
        hi = _log(rng, 1, 20000 if groups * width > 16 else 60000)
        return dict(op=op, G=rng.choice([1, 3, 4, 6, 8, 12, 16]), Hkv=rng.choice([1, 2, 4]),
                    sys=rng.choice([0, _log(rng, 1, 8000)]), groups=groups, width=width,
                    lo=rng.choice([1, max(1, hi // 2), hi]), hi=hi, tail=rng.choice([0, 1, _log(rng, 1, 1000)]),
                    empty=rng.choice([0, 0, 3]))
    if op == "select":
        W = _log(rng, 1, 16)
        V = _log(rng, 100, 131072)
        N = max(1, min(_log(rng, 1, 64), (1 << 25) // (W * V)))
        return dict(op=op, N=N, W=W, V=V, K=min(64, rng.choice([1, 2]) * W), bits=rng.choice([16, 32]),
                    pad=rng.choice([0, 0, rng.randrange(1, 64)]), masked=rng.choice([0.0, 0.0, 0.5]),
                    ended=rng.choice([0.0, 0.3]))
    if op == "reorder":
        B, per = _log(rng, 1, 1000), _log(rng, 1, 1024)
        return dict(op=op, B=B, width=rng.choice([1, 2, 4, 8, 16]), per_row=per, pages=B * per + rng.randrange(1, 500))
    hi = _log(rng, 1, 2000)
    return dict(op=op, S=_log(rng, 1, 8), lo=rng.choice([0, 1, hi]), hi=hi,
                before=rng.choice([0, rng.randrange(1, 3000)]), G=rng.choice([1, 4, 6, 16]),
                Hkv=rng.choice([1, 2, 4]), R=rng.choice([16, 32, 64, 128]),
                layout=rng.choice(["half", "interleaved"]),
                scaling=rng.choice(["none", "linear", "ntk", "yarn"]), norm=rng.random() < 0.75,
                index=rng.random() < 0.5)


# ------------------------------------------------------------------ sizes that follow from a case

def _blocks(x):
    return (x + BLOCK - 1) // BLOCK


def _attend_lens(c):
    """Per group the end of what its rows share, per row the length."""
    r = np.random.RandomState((c["lo"] * 1000003 + c["hi"] * 31 + c["groups"] * 7 + c["tail"]) % (1 << 31))
    shared = c["sys"] + r.randint(c["lo"], c["hi"] + 1, size=c["groups"])
    shared[0] = c["sys"] + c["hi"]
    lens = np.repeat(shared, c["width"]) + r.randint(0, c["tail"] + 1, size=c["groups"] * c["width"])
    if c["empty"]:
        lens[c["empty"] - 1::c["empty"]] = 0
    return shared, lens


def _append_lens(c):
    r = np.random.RandomState((c["lo"] * 1009 + c["hi"] * 31 + c["S"]) % (1 << 31))
    n = r.randint(c["lo"], c["hi"] + 1, size=c["S"])
    n[0] = max(1, n[0])
    return n


def _reorder_lens(c):
    r = np.random.RandomState(c["B"] * 131 + c["per_row"])
    return r.randint(0, c["per_row"] * BLOCK + 1, size=c["B"])


def work(c):
    op = c["op"]
    if op == "attend":
        shared, lens = _attend_lens(c)
        live = lens[lens > 0]
        rows = lens.reshape(c["groups"], c["width"])
        # tokens that some row reads, those of shared pages once
        sys = c["sys"] // BLOCK * BLOCK if len(live) > 1 else 0
        first = np.maximum(shared // BLOCK * BLOCK, sys) if c["width"] > 1 else np.full(c["groups"], sys)
        n = sys if len(live) else 0
        n += int(sum(f - sys for f, r in zip(first, rows) if (r > 0).any()))
        n += int(sum((r[r > 0] - f).sum() for f, r in zip(first, rows)))
        Hq, B = c["G"] * c["Hkv"], len(lens)
        return {"bytes": n * c["Hkv"] * 512 + B * Hq * (512 + 4) + 4 * (B + int(_blocks(live).sum())),
                "flops": 4 * D * Hq * int(live.sum())}
    if op == "select":
        n = c["N"] * c["W"] * c["V"]
        return {"bytes": n * c["bits"] // 8 + 5 * c["N"] * c["W"] + 12 * c["N"] * c["K"], "flops": 4 * n}
    if op == "reorder":
        n = int(_blocks(_reorder_lens(c)).sum())
        return {"bytes": 4 * (4 * n + 4 * c["B"]), "flops": n}
    T, Hkv = int(_append_lens(c).sum()), c["Hkv"]
    heads = c["G"] * Hkv + 2 * Hkv + 2 * Hkv * c["index"]
    return {"bytes": T * heads * 512 + 8 * c["S"], "flops": 10 * D * T * (heads - Hkv)}


# ------------------------------------------------------------------ inputs

def _randn(g, *shape, std=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std)


def _ints(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def _attend_table(c, rng):
    """Block table whose rows share the full pages of the system prompt and of their group's prompt."""
    shared, lens = _attend_lens(c)
    nb = _blocks(lens)
    table = np.full((len(lens), max(1, int(nb.max()))), -1, np.int64)
    at = 0

    def fresh(n):
        nonlocal at
        at += n
        return np.arange(at - n, at)
    sys = fresh(c["sys"] // BLOCK)
    for i, end in enumerate(shared):
        own_pages = fresh(end // BLOCK - len(sys))
        for b in range(i * c["width"], (i + 1) * c["width"]):
            if nb[b]:
                row = np.concatenate([sys, own_pages, fresh(nb[b] - end // BLOCK)])
                table[b, :nb[b]] = row
    perm = rng.permutation(max(1, at))
    return np.where(table >= 0, perm[table], -1), lens, max(1, at)


def _freqs(R, scaling, factor, orig):
    """Angle per position of each of the R / 2 pairs, and the gain of the rotated channels."""
    base = BASE * factor ** (R / (R - 2)) if scaling == "ntk" else BASE
    f = base ** (-2.0 * np.arange(R // 2) / R)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "yarn":   # by parts: pairs that turn often keep their angle
        turns = orig * f / (2 * math.pi)
        keep = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
        return f / factor * (1 - keep) + f * keep, 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _handle(c):
    """The rotation that a program keeps: the frequencies and the gain, or the package's handle."""
    factor = 1.0 if c["scaling"] == "none" else 4.0
    if own:
        import msa_block_sparse_gb300 as m
        return m.msa_rope(c["R"], BASE, layout=c["layout"], scaling=c["scaling"], factor=factor,
                          orig_len=32768)
    f, gain = _freqs(c["R"], c["scaling"], factor, 32768)
    return torch.tensor(f, dtype=torch.float64, device="cuda"), gain


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rng = np.random.RandomState(seed % (1 << 31))
    s = dict(c)
    op = c["op"]
    if op == "attend":
        table, lens, pages = _attend_table(c, rng)
        s["q"] = _randn(g, len(lens), c["G"] * c["Hkv"], D).to(torch.bfloat16)
        for n in ("k_cache", "v_cache"):
            s[n] = torch.empty(pages, c["Hkv"], BLOCK, D, dtype=torch.bfloat16, device="cuda")
            s[n].normal_(generator=g)
        s["table"], s["lens"] = _ints(table), _ints(lens)
        return s
    if op == "select":
        N, W, V = c["N"], c["W"], c["V"]
        x = _randn(g, N * W, V + c["pad"], std=3.0)
        if c["masked"]:
            x[torch.rand(x.shape, generator=g, device="cuda") < c["masked"]] = -math.inf
        s["logits"] = x.to(torch.bfloat16 if c["bits"] == 16 else torch.float32)[:, :V]
        s["scores"] = -_randn(g, N * W).abs() * 2 - 5
        s["finished"] = None
        if c["ended"]:
            s["finished"] = torch.rand(N * W, generator=g, device="cuda") < c["ended"]
        return s
    if op == "reorder":
        B, pages, maxp = c["B"], c["pages"], c["per_row"]
        lens = _reorder_lens(c)
        nb = _blocks(lens)
        perm = rng.permutation(pages)
        at = np.concatenate([[0], np.cumsum(nb)])
        cols = np.arange(maxp)
        table = np.where(cols < nb[:, None], perm[np.minimum(at[:-1, None] + cols, pages - 1)], -1)
        first = np.arange(B) // c["width"] * c["width"]
        parents = first + rng.randint(0, np.minimum(c["width"], B - first))
        parents[rng.rand(B) < 0.03] = -1
        ref = np.zeros(pages, np.int64)
        ref[table[table >= 0]] = 1
        # the tables in one buffer, so that a pass can start from them again
        sizes = [B * maxp, B, pages]
        offs = np.concatenate([[0], np.cumsum([(n + 63) // 64 * 64 for n in sizes])])
        flat = np.zeros(offs[-1], np.int64)
        for o, v in zip(offs, (table, lens, ref)):
            flat[o:o + v.size] = v.reshape(-1)
        s["parents"], s["meta0"] = _ints(parents), _ints(flat)
        s["meta"] = s["meta0"].clone()
        s["table"] = s["meta"][:sizes[0]].view(B, maxp)
        s["lens"] = s["meta"][offs[1]:offs[1] + B]
        s["ref"] = s["meta"][offs[2]:offs[2] + pages]
        return s
    n, Hkv = _append_lens(c), c["Hkv"]
    T, end = int(n.sum()), n + c["before"]
    pages = int(_blocks(end).sum())
    perm = rng.permutation(pages)
    at = np.concatenate([[0], np.cumsum(_blocks(end))])
    cols = np.arange(int(_blocks(end).max()))
    s["table"] = _ints(np.where(cols < _blocks(end)[:, None], perm[np.minimum(at[:-1, None] + cols, pages - 1)], -1))
    s["cu"], s["lens"] = _ints(np.concatenate([[0], np.cumsum(n)])), _ints(end)
    heads = dict(q=c["G"] * Hkv, k=Hkv, v=Hkv, q_idx=Hkv, k_idx=Hkv)
    for name, h in heads.items():
        s[name] = _randn(g, T, h, D).to(torch.bfloat16) if c["index"] or "idx" not in name else None
    for name, of in (("w_q", "q"), ("w_k", "k"), ("w_qi", "q_idx"), ("w_ki", "k_idx")):
        s[name] = _randn(g, D, std=0.1).to(torch.bfloat16) if c["norm"] and s[of] is not None else None
    for name, of in (("k_cache", "k"), ("v_cache", "v"), ("kidx_cache", "k_idx")):
        s[name] = None
        if s[of] is not None:
            s[name] = torch.zeros(pages, Hkv, BLOCK, D, dtype=torch.bfloat16, device="cuda")
    s["rope"] = _handle(c)
    return s


# ------------------------------------------------------------------ plain forms

def _attend(s):
    q, lens, table = s["q"], s["lens"].long(), s["table"].long().clamp(min=0)
    B, Hkv, n = q.shape[0], s["Hkv"], table.shape[1] * BLOCK

    def held(cache):                                                   # [B, Hkv, n, 128]
        return cache[table].float().permute(0, 2, 1, 3, 4).reshape(B, Hkv, n, D)
    z = q.float().view(B, Hkv, s["G"], D) @ held(s["k_cache"]).transpose(-1, -2) / math.sqrt(D)
    hidden = torch.arange(n, device="cuda") >= lens[:, None]
    z.masked_fill_(hidden[:, None, None], -math.inf)
    top = z.amax(-1, keepdim=True)
    p = (z - top.masked_fill(top == -math.inf, 0)).exp()
    total = p.sum(-1, keepdim=True)
    o = p @ held(s["v_cache"]) / total.clamp(min=1e-30)
    lse = top + total.log()
    return o.view(B, -1, D).to(torch.bfloat16), lse.view(B, -1)


def _select(s):
    N, W, K = s["N"], s["W"], s["K"]
    x = s["logits"].double()
    top = x.amax(-1, keepdim=True)
    top = top.masked_fill(top == -math.inf, 0)
    cand = s["scores"].double()[:, None] + (x - (top + (x - top).exp().sum(-1, keepdim=True).log()))
    cand.masked_fill_(x == -math.inf, -math.inf)
    if s["finished"] is not None:      # an ended beam goes on as it is, by token 0
        cand.masked_fill_(s["finished"][:, None], -math.inf)
        cand[:, 0] = torch.where(s["finished"], s["scores"].double(), cand[:, 0])
    best, at = cand.view(N, -1).sort(dim=-1, descending=True, stable=True)
    best, at = best[:, :K], at[:, :K]
    none = best == -math.inf
    parents = torch.arange(N, device="cuda")[:, None] * W + at // s["V"]
    return (best.float(), parents.masked_fill(none, -1).int(), (at % s["V"]).masked_fill(none, -1).int())


def _reorder(s):
    s["meta"].copy_(s["meta0"])
    table, lens, parents = s["table"].clone(), s["lens"].clone(), s["parents"].long()
    cols = torch.arange(table.shape[1], device="cuda")
    held = cols < ((lens + BLOCK - 1) // BLOCK)[:, None]
    after = torch.where(parents >= 0, lens[parents.clamp(min=0)], 0)
    keeps = cols < ((after + BLOCK - 1) // BLOCK)[:, None]
    to = torch.where(keeps, table[parents.clamp(min=0)], -1)
    change = torch.cat([torch.full_like(table[held], -1), torch.ones_like(to[keeps])])
    s["ref"].index_add_(0, torch.cat([table[held], to[keeps]]).long(), change)
    s["table"].copy_(to)
    s["lens"].copy_(after)
    return s["meta"], after.int()


def _prologue(s, x, w, cos, sin):
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * (1 + w.float())
    R = s["R"]
    if s["layout"] == "half":
        a, b = x[..., :R // 2], x[..., R // 2:R]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([y, x[..., R:]], -1).to(torch.bfloat16)


def _append(s):
    cu, f = s["cu"].long(), s["rope"]
    t = torch.arange(s["q"].shape[0], device="cuda")
    seq = torch.searchsorted(cu, t, right=True) - 1
    pos = s["lens"].long()[seq] - cu[seq + 1] + t
    angle = pos.double()[:, None, None] * f[0]
    cos, sin = (angle.cos() * f[1]).float(), (angle.sin() * f[1]).float()
    page, slot = s["table"][seq, pos // BLOCK].long(), pos % BLOCK
    s["k_cache"][page, :, slot] = _prologue(s, s["k"], s["w_k"], cos, sin)
    s["v_cache"][page, :, slot] = s["v"]
    q = _prologue(s, s["q"], s["w_q"], cos, sin)
    if not s["index"]:
        return q, s["k_cache"], s["v_cache"]
    s["kidx_cache"][page, :, slot] = _prologue(s, s["k_idx"], s["w_ki"], cos, sin)
    return q, s["k_cache"], s["v_cache"], _prologue(s, s["q_idx"], s["w_qi"], cos, sin), s["kidx_cache"]


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["op"]
    if not own:
        return {"attend": _attend, "select": _select, "reorder": _reorder, "append": _append}[op](s)
    import msa_block_sparse_gb300 as m
    if op == "attend":
        return m.msa_decode_shared(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"])
    if op == "select":
        return m.msa_beam_select(s["logits"], s["scores"], s["W"], s["K"], finished=s["finished"])
    if op == "reorder":
        s["meta"].copy_(s["meta0"])
        kept = m.msa_pages_reorder(s["parents"], s["table"], s["lens"], s["ref"])
        return s["meta"], kept
    q, qi = m.msa_cache_append(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["cu"],
                               s["lens"], s["rope"], w_q=s["w_q"], w_k=s["w_k"], q_idx=s["q_idx"],
                               k_idx=s["k_idx"], kidx_cache=s["kidx_cache"], w_qi=s["w_qi"], w_ki=s["w_ki"])
    if not s["index"]:
        return q, s["k_cache"], s["v_cache"]
    return q, s["k_cache"], s["v_cache"], qi, s["kidx_cache"]


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(c, seed):
    op = c["op"]
    if op == "reorder":
        return None                      # whole numbers: held to equality
    global own
    kept, own = own, False
    try:
        s = prepare(c, seed)
    finally:
        own = kept
    if op == "attend":
        lens, G = s["lens"].tolist(), c["G"]
        o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        lse = torch.full(o.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
        for b, L in enumerate(lens):
            if L == 0:
                continue
            pages = s["table"][b, :_blocks(L)].long()
            for h in range(c["Hkv"]):
                k = s["k_cache"][pages, h].reshape(-1, D)[:L].double()
                v = s["v_cache"][pages, h].reshape(-1, D)[:L].double()
                x = torch.mm(s["q"][b, h * G:(h + 1) * G].double(), k.t()) * D ** -0.5
                lse[b, h * G:(h + 1) * G] = torch.logsumexp(x, 1)
                o[b, h * G:(h + 1) * G] = torch.softmax(x, 1) @ v
        return o, lse
    if op == "select":
        best = torch.full((c["N"], c["K"]), -math.inf, dtype=torch.float64, device="cuda")
        for n in range(c["N"]):
            found = []
            for w in range(n * c["W"], (n + 1) * c["W"]):
                if s["finished"] is not None and bool(s["finished"][w]):
                    found.append(s["scores"][w:w + 1].double())
                    continue
                x = torch.log_softmax(s["logits"][w].double(), 0) + s["scores"][w].double()
                x = x[torch.isfinite(x)]
                found.append(x.topk(min(c["K"], x.numel()))[0])
            found = torch.cat(found).sort(descending=True)[0][:c["K"]]
            best[n, :found.numel()] = found
        return best, None, None
    f, gain = s["rope"]
    n = _append_lens(c)
    pos = torch.cat([torch.arange(c["before"], c["before"] + int(m)) for m in n]).cuda()
    row = torch.repeat_interleave(torch.arange(c["S"]), torch.as_tensor(n)).cuda()
    turn = torch.polar(torch.full((pos.numel(), 1, f.numel()), gain, dtype=torch.float64, device="cuda"),
                       pos.double()[:, None, None] * f)
    R = c["R"]

    def turned(x, w):
        y = x.double()
        if w is not None:
            y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS) * (w.double() + 1)
        first, second = (slice(0, R // 2), slice(R // 2, R)) if c["layout"] == "half" else (slice(0, R, 2), slice(1, R, 2))
        z = torch.complex(y[..., first], y[..., second]) * turn
        y = y.clone()
        y[..., first], y[..., second] = z.real, z.imag
        return y

    def paged(x):
        out = torch.zeros(s["k_cache"].shape, dtype=torch.float64, device="cuda")
        out[s["table"].long()[row, pos // BLOCK], :, pos % BLOCK] = x
        return out
    out = [turned(s["q"], s["w_q"]), paged(turned(s["k"], s["w_k"])), paged(s["v"].double())]
    if c["index"]:
        out += [turned(s["q_idx"], s["w_qi"]), paged(turned(s["k_idx"], s["w_ki"]))]
    return tuple(out)


if __name__ == "__main__":
    for case in listed() + [draw(random.Random(i)) for i in range(4)]:
        print(case, work(case))
