"""The operators of a long-context serving and training path beside the block-sparse
attention: the normed and rotated queries and keys (any rotary layout, part of the
head, frequencies scaled for long contexts), a paged cache held in 4 bits with the
decode step that reads it, and the upkeep of the cache's pages.

`run` computes each operator in plain torch operations (32 bits, 64 for angles and
for block scores, whose order decides a selection), or, where `own` is true, by the
calls of this repository's package.

The 4-bit format: 16 consecutive channels of a token share one scale (e4m3, the
largest magnitude / 6 rounded to nearest even), each value is the nearest e2m1
number (0, 0.5, 1, 1.5, 2, 3, 4, 6 with a sign, ties to the even code) of value /
scale; a page of one head holds 128 tokens: 128 x 64 bytes of codes (low nibble =
even channel), then 128 x 8 bytes of scales.
"""
import math
import random

import numpy as np
import torch

own = False

BLOCK, TOPK, D4, SLAB = 128, 16, 128, 128 * 72
BASE, EPS = 1.0e7, 1.0e-6
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # q of one decode step of 32 sequences, positions far beyond the trained length
        dict(name="rotate-decode-32", op="rotate", T=32, H=64, D=128, R=64, layout="half",
             scaling="yarn", factor=8.0, norm=True, far=120000),
        # the 64 query heads of a 16k-token pack
        dict(name="rotate-pack-16k", op="rotate", T=16384, H=64, D=128, R=64, layout="half",
             scaling="yarn", factor=4.0, norm=True, far=0),
        # training: gradients of the 12 query heads of head dim 256, whole head rotated
        dict(name="rotate-grad-d256", op="rotate_bwd", T=16384, H=12, D=256, R=256,
             layout="interleaved", scaling="linear", factor=2.0, norm=True, far=0),
        # the new token of 64 sequences: norms, rotation, 4-bit store
        dict(name="append-b64", op="append", B=64, G=16, Hkv=4, lo=8192, hi=32768),
        # a prefill pack of 8 sequences into the 4-bit cache and back
        dict(name="store-pack-16k", op="store", S=8, Hkv=4, lo=512, hi=4096, start=0),
        # a chunk of a chunked prefill: 5 short pieces at odd positions
        dict(name="store-chunk", op="store", S=5, Hkv=2, lo=1, hi=150, start=777),
        # one user, short context: latency
        dict(name="decode-b1-short", op="decode", B=1, G=16, Hkv=4, lo=1500, hi=1500, n_init=0),
        # the serving batch of the framework's benchmark
        dict(name="decode-b64", op="decode", B=64, G=16, Hkv=4, lo=8192, hi=32768, n_init=0),
        # few users with very long contexts, first block always kept
        dict(name="decode-b5-long", op="decode", B=5, G=16, Hkv=4, lo=60000, hi=131000, n_init=1),
        # 6 query heads per KV head, empty and one-token rows among the lengths
        dict(name="decode-b33-g6", op="decode", B=33, G=6, Hkv=2, lo=0, hi=9000, n_init=0),
        # beam search: every live row forked, then all rows take one token
        dict(name="branch-48", op="branch", B=96, Hkv=4, pages=1536, per_row=24),
        # half the rows end, the pool is packed to its front
        dict(name="compact-4096", op="compact", B=128, Hkv=1, pages=4096, per_row=40),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "rotate_bwd", "append", "store", "decode", "decode", "branch",
                     "compact"])
    if op in ("rotate", "rotate_bwd"):
        D = rng.choice([64, 128, 256])
        H = rng.choice([1, 2, 4, 5, 12, 16, 24, 64])
        T = min(_log(rng, 1, 16384), (1 << (27 if op == "rotate" else 26)) // (H * D))
        return dict(op=op, T=T, H=H, D=D, R=rng.choice([r for r in (16, 32, 64, 96, 128, 256) if r <= D]),
                    layout=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "linear", "ntk", "yarn"]),
                    factor=rng.choice([2.0, 4.0, 8.0]), norm=rng.random() < 0.75,
                    far=rng.choice([0, rng.randrange(1, 1000000)]))
    if op == "append":
        return dict(op=op, B=_log(rng, 1, 64), G=rng.choice([1, 4, 6, 8, 16]),
                    Hkv=rng.choice([1, 2, 4]), lo=1, hi=_log(rng, 1, 32768))
    if op == "store":
        hi = _log(rng, 1, 2200)
        return dict(op=op, S=_log(rng, 1, 8), Hkv=rng.choice([1, 2, 3, 4]), lo=rng.randrange(0, hi + 1),
                    hi=hi, start=rng.choice([0, rng.randrange(0, 3000)]))
    if op == "decode":
        B, Hkv = _log(rng, 1, 64), rng.choice([1, 2, 4])
        hi = _log(rng, 1, 20000 if B > 8 else 131000)
        return dict(op=op, B=B, G=rng.choice([1, 3, 6, 8, 12, 16]), Hkv=Hkv,
                    lo=rng.choice([hi, hi // 2, 0]), hi=hi, n_init=rng.choice([0, 0, 1, 4, 15]))
    if op == "branch":
        B = 2 * _log(rng, 1, 64)
        per = _log(rng, 1, 24)
        return dict(op=op, B=B, Hkv=rng.choice([1, 2, 4]), pages=B * per + rng.randrange(0, 200),
                    per_row=per)
    B = _log(rng, 2, 128)
    per = _log(rng, 1, 28)
    return dict(op=op, B=B, Hkv=1, pages=B * per + rng.randrange(0, 300), per_row=per)


# ------------------------------------------------------------------ sizes that follow from a case

def _lens(c, n):
    """n lengths in [lo, hi] that belong to the case, both ends among them when n > 2."""
    r = np.random.RandomState((c["lo"] * 1000003 + c["hi"] * 31 + n) % (1 << 31))
    x = r.randint(c["lo"], c["hi"] + 1, size=n)
    if n > 2:
        x[0], x[1] = c["hi"], c["lo"]
    return x.astype(np.int64)


def _branch_lens(c):
    """The live half of the rows hold 1 .. per_row pages (the other half is empty)."""
    n = c["B"] // 2
    r = np.random.RandomState(c["B"] * 131 + c["per_row"])
    return r.randint(1, c["per_row"] * BLOCK + 1, size=n).astype(np.int64)


def _compact_lens(c):
    r = np.random.RandomState(c["B"] * 137 + c["per_row"])
    return r.randint(0, c["per_row"] * BLOCK + 1, size=c["B"]).astype(np.int64)


def _blocks(x):
    return (x + BLOCK - 1) // BLOCK


def work(c):
    op = c["op"]
    if op in ("rotate", "rotate_bwd"):
        n = c["T"] * c["H"] * c["D"]
        pos = 4 * c["T"] if c["far"] else 8
        if op == "rotate":
            return {"bytes": 4 * n + 2 * c["D"] * c["norm"] + pos, "flops": 8 * n}
        return {"bytes": 2 * n * (3 if c["norm"] else 2) + 6 * c["D"] * c["norm"] + pos,
                "flops": 16 * n}
    if op == "append":
        row = c["B"] * c["Hkv"]
        q = row * c["G"] * 256 + row * 256
        return {"bytes": 2 * q + 3 * row * (256 + 72 + 72 + 256) + 8 * c["B"],
                "flops": 10 * 128 * row * (c["G"] + 4)}
    if op == "store":
        rows = int(_lens(c, c["S"]).sum()) * c["Hkv"] * 3
        return {"bytes": max(1, rows * (256 + 72 + 72 + 256)), "flops": 12 * 128 * rows}
    if op == "decode":
        L = _lens(c, c["B"])
        nb = _blocks(L)
        scored = np.where(nb > TOPK, np.maximum(nb - 1 - c["n_init"], 0), 0)
        keys = np.minimum(nb, TOPK) * BLOCK - (nb * BLOCK - L)   # the own block may be partial
        row = c["B"] * c["Hkv"]
        b = c["Hkv"] * (int(scored.sum()) * SLAB + int(keys.sum()) * 144) \
            + row * (c["G"] * 512 + 256 + 64)
        f = c["Hkv"] * (int(scored.sum()) * BLOCK * 256 + int(keys.sum()) * 512 * c["G"])
        return {"bytes": b, "flops": f}
    page = c["Hkv"] * BLOCK * D4 * 2 * 3
    if op == "branch":
        L = _branch_lens(c)
        moved = 2 * int((L % BLOCK != 0).sum())
        meta = 4 * (int(_blocks(L).sum()) * 3 + 2 * c["B"] + c["pages"])
        return {"bytes": 2 * moved * page + meta, "flops": c["pages"]}
    L = _compact_lens(c)
    live = int(_blocks(L[1::2]).sum())
    moved = live * (c["pages"] - live) / c["pages"]
    return {"bytes": 2 * moved * page + 4 * (3 * c["pages"] + 2 * live), "flops": c["pages"]}


# ------------------------------------------------------------------ inputs

def _randn(g, *shape, std=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std)


def _ints(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def _table(rng, lens, max_pages, pages):
    """Block table of rows with these lengths over a shuffled pool."""
    nb = _blocks(np.asarray(lens))
    perm = rng.permutation(pages)
    t = np.full((len(lens), max_pages), -1, np.int32)
    at = 0
    for b, n in enumerate(nb):
        t[b, :n] = perm[at:at + n]
        at += n
    return t


def _pool4(g, pages, heads, offsets):
    """A pool of 4-bit pages of normal values (index keys: one offset per block)."""
    out = torch.empty(pages, heads, SLAB, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 27) // (heads * BLOCK * D4))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        x = _randn(g, n, heads, BLOCK, D4)
        if offsets:
            x += _randn(g, n, heads, 1, D4, std=0.5)
        out[p:p + n] = _slab(*_quantise(x.to(torch.bfloat16).float()))
    return out


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rng = np.random.RandomState(seed % (1 << 31))
    s = dict(c)
    op = c["op"]
    if op in ("rotate", "rotate_bwd"):
        T, H, D = c["T"], c["H"], c["D"]
        s["x"] = _randn(g, T, H, D).to(torch.bfloat16)
        s["w"] = _randn(g, D, std=0.1).to(torch.bfloat16) if c["norm"] else None
        if op == "rotate_bwd":
            s["dy"] = _randn(g, T, H, D).to(torch.bfloat16)
        s["positions"] = s["cu"] = None
        if c["far"]:
            s["positions"] = _ints(rng.randint(0, c["far"] + 1, size=T))
        else:
            cuts = np.sort(rng.randint(0, T + 1, size=3))
            s["cu"] = _ints(np.concatenate([[0], cuts, [T]]))
        s["rope"] = _handle(c)
        return s
    if op == "append":
        B, Hkv, Hq = c["B"], c["Hkv"], c["G"] * c["Hkv"]
        L = np.maximum(_lens(c, B), 1)
        pages = int(_blocks(L).sum())
        for n, h in (("q", Hq), ("q_idx", Hkv), ("k", Hkv), ("v", Hkv), ("k_idx", Hkv)):
            s[n] = _randn(g, B, h, D4).to(torch.bfloat16)
        for n in ("w_q", "w_qi", "w_k", "w_ki"):
            s[n] = _randn(g, D4, std=0.1).to(torch.bfloat16)
        s["caches"] = [torch.zeros(pages, Hkv, SLAB, dtype=torch.uint8, device="cuda") for _ in range(3)]
        s["table"] = _ints(_table(rng, L, int(_blocks(L).max()), pages))
        s["lens"] = _ints(L)
        s["before"] = _ints(L - 1)
        s["cu"] = _ints(np.arange(B + 1))
        s["rope"] = _handle(dict(R=64, layout="half", scaling="yarn", factor=4.0))
        return s
    if op == "store":
        S, Hkv = c["S"], c["Hkv"]
        L = _lens(c, S)
        if int(L.sum()) == 0:
            L[0] = 1
        T, end = int(L.sum()), L + c["start"]
        pages = int(_blocks(end).sum())
        off = _randn(g, T // BLOCK + 1, Hkv, D4, std=0.5).repeat_interleave(BLOCK, 0)[:T]
        s["k"] = _randn(g, T, Hkv, D4).to(torch.bfloat16)
        s["v"] = _randn(g, T, Hkv, D4).to(torch.bfloat16)
        s["k_idx"] = (_randn(g, T, Hkv, D4) + off).to(torch.bfloat16)
        s["caches"] = [torch.zeros(pages, Hkv, SLAB, dtype=torch.uint8, device="cuda") for _ in range(3)]
        s["table"] = _ints(_table(rng, end, int(_blocks(end).max()), pages))
        s["cu"] = _ints(np.concatenate([[0], np.cumsum(L)]))
        s["first"] = _ints(np.full(S, c["start"]))
        return s
    if op == "decode":
        B, Hkv, Hq = c["B"], c["Hkv"], c["G"] * c["Hkv"]
        L = _lens(c, B)
        pages = max(1, int(_blocks(L).sum()))
        s["q"] = _randn(g, B, Hq, D4).to(torch.bfloat16)
        s["q_idx"] = _randn(g, B, Hkv, D4).to(torch.bfloat16)
        s["caches"] = [_pool4(g, pages, Hkv, offsets=n == 2) for n in range(3)]
        s["table"] = _ints(_table(rng, L, max(1, int(_blocks(L).max())), pages))
        s["lens"] = _ints(L)
        if own:
            import msa_block_sparse_gb300 as m
            s["ws"] = torch.empty(m.workspace_bytes("decode4_step", B, Hq, Hkv, s["table"].shape[1]),
                                  dtype=torch.uint8, device="cuda")
        return s
    # page upkeep: the tables in one buffer, so that a pass can start from them again
    B, pages = c["B"], c["pages"]
    L = np.zeros(B, np.int64)
    if op == "branch":
        L[:B // 2] = _branch_lens(c)
        src = rng.randint(0, B // 2, size=B // 2)
        s["src"], s["dst"] = _ints(src), _ints(np.arange(B // 2, B))
        s["add"] = _ints(np.ones(B))
    else:
        L[:] = _compact_lens(c)
        s["rows"] = _ints(np.arange(0, B, 2))
    maxp = c["per_row"] + 1
    table = _table(rng, L, maxp, pages)
    ref = np.zeros(pages, np.int32)
    ref[table[table >= 0]] = 1
    sizes = [B * maxp, B, pages]
    at, offs = 0, []
    for n in sizes:
        offs.append(at)
        at += (n + 63) // 64 * 64
    flat = np.zeros(at, np.int32)
    for o, v in zip(offs, (table, L, ref)):
        flat[o:o + v.size] = v.reshape(-1)
    s["meta0"] = _ints(flat)
    s["meta"] = s["meta0"].clone()
    s["table"] = s["meta"][:sizes[0]].view(B, maxp)
    s["lens"] = s["meta"][offs[1]:offs[1] + B]
    s["ref"] = s["meta"][offs[2]:offs[2] + pages]
    s["caches"] = [_randn(g, pages, c["Hkv"], BLOCK, D4).to(torch.bfloat16) for _ in range(3)]
    return s


def _handle(c):
    """The rotation that a program keeps: the frequencies and the gain, or the package's handle."""
    if own:
        import msa_block_sparse_gb300 as m
        return m.msa_rope(c["R"], BASE, layout=c["layout"], scaling=c["scaling"],
                          factor=c["factor"], orig_len=32768)
    f, gain = _freqs(c["R"], c["scaling"], c["factor"], 32768)
    return torch.tensor(f, dtype=torch.float64, device="cuda"), gain


def _freqs(R, scaling, factor, orig):
    """Angle per position of each of the R / 2 pairs, and the gain of the rotated channels."""
    base = BASE * factor ** (R / (R - 2)) if scaling == "ntk" else BASE
    f = np.array([base ** (-2.0 * i / R) for i in range(R // 2)])
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "yarn":   # by parts: pairs that turn often keep their angle
        turns = orig * f / (2 * math.pi)
        keep = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
        return f / factor * (1 - keep) + f * keep, 0.1 * math.log(factor) + 1.0
    return f, 1.0


# ------------------------------------------------------------------ plain forms

def _positions(s, T):
    if s["positions"] is not None:
        return s["positions"].long()
    t = torch.arange(T, device="cuda")
    cu = s["cu"].long()
    seq = (t[:, None] >= cu[None, 1:-1]).sum(1)
    return t - cu[seq]


def _cos_sin(pos, rope):
    f, gain = rope
    a = pos.double()[:, None] * f
    return (a.cos() * gain).float()[:, None], (a.sin() * gain).float()[:, None]


def _turn(z, cos, sin, R, layout):
    """The first R channels of z [T, H, D] turned by the angles."""
    if layout == "half":
        a, b = z[..., :R // 2], z[..., R // 2:R]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = z[..., 0:R:2], z[..., 1:R:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([y, z[..., R:]], -1)


def _normed(x, w):
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    return x * r * (1 + w)


def _prologue(x, w, pos, rope, R=64, layout="half"):
    z = x.float() if w is None else _normed(x.float(), w.float())
    return _turn(z, *_cos_sin(pos, rope), R, layout).to(torch.bfloat16)


def _prologue_grad(s):
    x, dy = s["x"].float(), s["dy"].float()
    cos, sin = _cos_sin(_positions(s, s["T"]), s["rope"])
    dz = _turn(dy, cos, -sin, s["R"], s["layout"])
    if s["w"] is None:
        return dz.to(torch.bfloat16)
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    xh, gz = x * r, dz * (1 + s["w"].float())
    dx = r * (gz - xh * (gz * xh).mean(-1, keepdim=True))
    return dx.to(torch.bfloat16), (dz * xh).double().sum((0, 1)).float()


def _quantise(x):
    """x [..., 128] -> codes uint8 [..., 64] and scale bytes uint8 [..., 8]."""
    b = x.unflatten(-1, (8, 16))
    s8 = (b.abs().amax(-1) / 6).clamp(max=448.0).to(torch.float8_e4m3fn)
    sc = s8.float()[..., None]
    m = torch.where(sc > 0, b.abs() / sc, torch.zeros_like(b))
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5)
            + (m >= 3.5) + (m > 5))
    code = (code + 8 * (b < 0)).to(torch.uint8).flatten(-2)
    bad = ~b.isfinite().all(-1)
    return (code[..., 0::2] | (code[..., 1::2] << 4),
            torch.where(bad, torch.full_like(s8.view(torch.uint8), 127), s8.view(torch.uint8)))


def _slab(codes, scales):
    """[..., 128, 64] and [..., 128, 8] -> [..., 9216]"""
    return torch.cat([codes.flatten(-2), scales.flatten(-2)], -1)


def _values(codes, scales):
    lut = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device="cuda")
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()
    return lut[n].unflatten(-1, (8, 16)).mul_(scales.view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)


def _page_values(slab):
    """[..., 9216] -> [..., 128, 128]"""
    return _values(slab[..., :8192].unflatten(-1, (128, 64)), slab[..., 8192:].unflatten(-1, (128, 8)))


def _where(s, seq, pos):
    """Page and slot of each token of rows `seq` at positions `pos`."""
    return s["table"][seq, pos // BLOCK].long(), pos % BLOCK


def _rows_in(cache, page, slot, x):
    codes, scales = _quantise(x)
    cache[:, :, :8192].unflatten(-1, (128, 64))[page, :, slot] = codes
    cache[:, :, 8192:].unflatten(-1, (128, 8))[page, :, slot] = scales


def _rows_out(cache, page, slot):
    return _values(cache[:, :, :8192].unflatten(-1, (128, 64))[page, :, slot],
                   cache[:, :, 8192:].unflatten(-1, (128, 8))[page, :, slot]).to(torch.bfloat16)


def _append(s):
    b = torch.arange(s["B"], device="cuda")
    pos = s["lens"].long() - 1
    page, slot = _where(s, b, pos)
    q = _prologue(s["q"], s["w_q"], pos, s["rope"])
    qi = _prologue(s["q_idx"], s["w_qi"], pos, s["rope"])
    k = _prologue(s["k"], s["w_k"], pos, s["rope"])
    ki = _prologue(s["k_idx"], s["w_ki"], pos, s["rope"])
    kc, vc, ic = s["caches"]
    _rows_in(kc, page, slot, k.float())
    _rows_in(vc, page, slot, s["v"].float())
    _rows_in(ic, page, slot, ki.float())
    return q, qi, _rows_out(kc, page, slot), _rows_out(vc, page, slot), _rows_out(ic, page, slot)


def _store(s):
    T = s["k"].shape[0]
    t = torch.arange(T, device="cuda")
    cu = s["cu"].long()
    seq = (t[:, None] >= cu[None, 1:-1]).sum(1)
    page, slot = _where(s, seq, t - cu[seq] + s["first"].long()[seq])
    kc, vc, ic = s["caches"]
    _rows_in(kc, page, slot, s["k"].float())
    _rows_in(vc, page, slot, s["v"].float())
    _rows_in(ic, page, slot, s["k_idx"].float())
    return _rows_out(kc, page, slot), _rows_out(vc, page, slot), _rows_out(ic, page, slot)


def _decode(s):
    B, G, Hkv = s["B"], s["G"], s["Hkv"]
    kc, vc, ic = s["caches"]
    L, table = s["lens"].long(), s["table"].long()
    n = table.shape[1]
    own_block = (L + BLOCK - 1) // BLOCK - 1
    blk = torch.arange(n, device="cuda")
    # every block's largest index logit, in 64 bits: near scores decide a selection
    idx = _page_values(ic[table.clamp(min=0)]).double()                     # [B, n, Hkv, 128, 128]
    score = (idx * s["q_idx"].double()[:, None, :, None, :]).sum(-1).amax(-1)
    score = score.transpose(1, 2)                                           # [B, Hkv, n]
    score = torch.where(blk < s["n_init"], math.inf, score)
    own_b = own_block[:, None, None]
    score = torch.where(blk >= own_b, -math.inf, score)
    order = score.sort(dim=-1, descending=True, stable=True).indices[..., :TOPK - 1]
    kept = torch.where(order < own_b, order, n)
    sel = torch.cat([kept, torch.where(own_b >= 0, own_b, n).expand(B, Hkv, 1)], -1).sort(-1).values
    if sel.shape[-1] < TOPK:
        sel = torch.cat([sel, torch.full((B, Hkv, TOPK - sel.shape[-1]), n, device="cuda")], -1)
    have = sel < n
    sel = torch.where(have, sel, 0)
    page = table.gather(1, sel.flatten(1)).view_as(sel).clamp(min=0)
    head = torch.arange(Hkv, device="cuda")[None, :, None]
    K, V = _page_values(kc[page, head]).flatten(2, 3), _page_values(vc[page, head]).flatten(2, 3)
    pos = sel[..., None] * BLOCK + torch.arange(BLOCK, device="cuda")
    ok = (have[..., None] & (pos < L[:, None, None, None])).flatten(2)      # [B, Hkv, 2048]
    q = s["q"].float().view(B, Hkv, G, D4)
    z = (q @ K.transpose(-1, -2)) / math.sqrt(D4)
    z = torch.where(ok[:, :, None], z, -math.inf)
    top = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(top.isinf(), 0.0, top))
    o = (p @ torch.where(ok[..., None], V, 0.0)) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    return o.view(B, Hkv * G, D4).to(torch.bfloat16), torch.where(have, sel, -1).int()


def _branch(s):
    s["meta"].copy_(s["meta0"])
    table, lens, ref = s["table"], s["lens"], s["ref"]
    src, dst = s["src"].long(), s["dst"].long()
    n = table.shape[1]
    col = torch.arange(n, device="cuda")
    # fork: the children share every page of their parents
    table[dst] = torch.where(col < _blocks(lens[src])[:, None], table[src], table[dst])
    lens[dst] = lens[src]
    shared = table[dst][col < _blocks(lens[dst])[:, None]].long()
    ref.index_add_(0, shared, torch.ones_like(shared, dtype=torch.int32))
    # extend: one token each; a shared last page that is not full is copied first
    old, new = lens.long(), lens.long() + s["add"].long()
    last = table.gather(1, (_blocks(old) - 1).clamp(min=0)[:, None])[:, 0].long()
    cow = (old % BLOCK != 0) & (s["add"] > 0) & (ref[last.clamp(min=0)] > 1)
    fresh = _blocks(new) - _blocks(old)
    need = fresh + cow
    at = need.cumsum(0) - need
    free = (ref == 0).nonzero()[:, 0]
    done = ((at + need <= free.numel()) | (need == 0)) & (new <= n * BLOCK)
    cow, fresh = cow & done, torch.where(done, fresh, 0)
    free = torch.cat([free, free.new_zeros(1)])
    first = free[at.clamp(max=free.numel() - 1)]
    rows = cow.nonzero()[:, 0]
    for_copy, to = last[rows], first[rows]
    ref.index_add_(0, for_copy, -torch.ones_like(for_copy, dtype=torch.int32))
    ref[to] = 1
    table[rows, _blocks(old)[rows] - 1] = to.int()
    grown = (fresh > 0).nonzero()[:, 0]          # one token: at most one fresh page
    page = free[(at + cow)[grown]]
    ref[page] = 1
    table[grown, _blocks(old)[grown]] = page.int()
    lens.copy_(torch.where(done, new, old))
    for_each = [cache.index_copy_(0, to, cache[for_copy]) for cache in s["caches"]]
    return [s["meta"], done.int()] + [cache.view(torch.int16) for cache in for_each]


def _compact(s):
    s["meta"].copy_(s["meta0"])
    table, lens, ref = s["table"], s["lens"], s["ref"]
    rows = s["rows"].long()
    col = torch.arange(table.shape[1], device="cuda")
    # free the rows that end
    held = col < _blocks(lens[rows])[:, None]
    gone = table[rows][held].long()
    ref.index_add_(0, gone, -torch.ones_like(gone, dtype=torch.int32))
    table[rows] = torch.where(held, -1, table[rows])
    lens[rows] = 0
    # pack the live pages to the front: those behind go to the free places, both ascending
    live = ref > 0
    n_live = live.sum()
    p = torch.arange(s["pages"], device="cuda")
    src, dst = (live & (p >= n_live)).nonzero()[:, 0], (~live & (p < n_live)).nonzero()[:, 0]
    where_to = torch.where(live, p, -1)
    where_to[src] = dst
    ref[dst] = ref[src]
    ref[src] = 0
    held = col < _blocks(lens)[:, None]
    table.copy_(torch.where(held, where_to[table.clamp(min=0).long()].int(), table))
    packed = [cache.index_copy_(0, dst, cache[src]) for cache in s["caches"]]
    return [s["meta"], where_to.int(), n_live.int().view(1)] + [cache.view(torch.int16) for cache in packed]


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["op"]
    if not own:
        if op == "rotate":
            return _prologue(s["x"], s["w"], _positions(s, s["T"]), s["rope"], s["R"], s["layout"])
        if op == "rotate_bwd":
            return _prologue_grad(s)
        return {"append": _append, "store": _store, "decode": _decode, "branch": _branch,
                "compact": _compact}[op](s)
    import msa_block_sparse_gb300 as m
    if op == "rotate":
        return m.msa_qk_norm_rope_ex(s["x"], s["w"], s["rope"], cu_seqlens=s["cu"],
                                     positions=s["positions"])
    if op == "rotate_bwd":
        dx, dw = m.msa_qk_norm_rope_bwd_ex(s["x"], s["dy"], s["w"], s["rope"], cu_seqlens=s["cu"],
                                           positions=s["positions"])
        return dx if s["w"] is None else (dx, dw)
    if op == "append":
        q, qi = m.msa_decode4_append(s["q"], s["q_idx"], s["k"], s["v"], s["k_idx"], s["w_q"],
                                     s["w_qi"], s["w_k"], s["w_ki"], *s["caches"], s["table"],
                                     s["lens"], s["rope"])
        return (q, qi) + m.msa_cache4_load(*s["caches"], s["table"], s["cu"], s["B"], start=s["before"])
    if op == "store":
        m.msa_cache4_store(s["k"], s["v"], s["k_idx"], *s["caches"], s["table"], s["cu"],
                           start=s["first"])
        return m.msa_cache4_load(*s["caches"], s["table"], s["cu"], s["k"].shape[0], start=s["first"])
    if op == "decode":
        return m.msa_decode4_step(s["q"], s["q_idx"], *s["caches"], s["table"], s["lens"],
                                  workspace=s["ws"], n_init=s["n_init"])
    s["meta"].copy_(s["meta0"])
    if op == "branch":
        m.msa_pages_fork(s["src"], s["dst"], s["table"], s["lens"], s["ref"])
        done = m.msa_pages_extend(s["add"], s["table"], s["lens"], s["ref"], s["caches"])
        return [s["meta"], done] + [cache.view(torch.int16) for cache in s["caches"]]
    m.msa_pages_free(s["rows"], s["table"], s["lens"], s["ref"])
    page_map, n_live = m.msa_pages_compact(s["table"], s["lens"], s["ref"], s["caches"])
    return [s["meta"], page_map, n_live] + [cache.view(torch.int16) for cache in s["caches"]]


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(c, seed):
    op = c["op"]
    if op in ("branch", "compact"):
        return None                      # moved bits: held to equality
    global own
    kept, own = own, False
    try:
        s = prepare(c, seed)
    finally:
        own = kept
    f, gain = s.get("rope", (None, 1.0))

    def turned(z, pos, sign=1.0):
        """Pairs as complex numbers times gain e^(i angle)."""
        R = 2 * f.numel()
        turn = torch.polar(torch.full((pos.numel(), f.numel()), gain, dtype=torch.float64, device="cuda"),
                           sign * pos.double()[:, None] * f[None])[:, None]
        y = z.clone()
        if c.get("layout", "half") == "half":
            t = torch.complex(z[..., :R // 2], z[..., R // 2:R]) * turn
            y[..., :R // 2], y[..., R // 2:R] = t.real, t.imag
        else:
            t = torch.complex(z[..., 0:R:2], z[..., 1:R:2]) * turn
            y[..., 0:R:2], y[..., 1:R:2] = t.real, t.imag
        return y

    def normed(x, w):
        x = x.double()
        return x / (x.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * (w.double() + 1)

    if op in ("rotate", "rotate_bwd"):
        if s["positions"] is not None:
            pos = s["positions"].double()
        else:
            cu = s["cu"].tolist()
            pos = torch.cat([torch.arange(b - a) for a, b in zip(cu, cu[1:])]).cuda().double()
        if op == "rotate":
            z = s["x"].double() if s["w"] is None else normed(s["x"], s["w"])
            return turned(z, pos)
        dz = turned(s["dy"].double(), pos, -1.0)
        if s["w"] is None:
            return dz
        x = s["x"].double()
        n = (x.pow(2).mean(-1, keepdim=True) + EPS).sqrt()
        gz = dz * (s["w"].double() + 1)
        return gz / n - x * (gz * x).mean(-1, keepdim=True) / n.pow(3), (dz * x / n).sum((0, 1))

    def four(x):
        """The value that 4 bits hold for x [..., 128], by the nearest of all codes."""
        b = x.reshape(*x.shape[:-1], 8, 16)
        e4 = torch.arange(127, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).double()
        want = b.abs().amax(-1) / 6

        def nearest(v, levels):
            hi = torch.searchsorted(levels, v.contiguous()).clamp(max=levels.numel() - 1)
            lo = (hi - 1).clamp(min=0)
            up, down = levels[hi] - v, v - levels[lo]
            return torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)

        scale = e4[nearest(want, e4)][..., None]
        lv = torch.tensor(LEVELS, dtype=torch.float64, device="cuda")
        m = torch.where(scale > 0, b.abs() / scale.clamp(min=1e-30), 0.0)
        return (torch.sign(b) * lv[nearest(m, lv)] * scale).reshape(x.shape)

    if op == "append":
        pos = s["lens"].double() - 1
        pre = [turned(normed(s[n], s[w]), pos) for n, w in (("q", "w_q"), ("q_idx", "w_qi"),
                                                            ("k", "w_k"), ("k_idx", "w_ki"))]
        held = [four(x.to(torch.bfloat16).double()) for x in (pre[2], s["v"], pre[3])]
        return pre[0], pre[1], held[0], held[1], held[2]
    if op == "store":
        return tuple(four(s[n].double()) for n in ("k", "v", "k_idx"))
    # decode: one sequence at a time
    lv = torch.tensor(LEVELS, dtype=torch.float64, device="cuda")

    def page(cache, p):
        raw = cache[p].long()                                           # [n, Hkv, 9216]
        byte, sc = raw[..., :8192].reshape(*raw.shape[:2], 128, 64), raw[..., 8192:].reshape(*raw.shape[:2], 128, 8)
        x = torch.empty(*raw.shape[:2], 128, 128, dtype=torch.float64, device="cuda")
        x[..., 0::2] = lv[byte & 7] * (1 - 2 * ((byte >> 3) & 1))
        x[..., 1::2] = lv[(byte >> 4) & 7] * (1 - 2 * (byte >> 7))
        e, mant = sc >> 3, (sc & 7).double()
        size = torch.where(e > 0, (8 + mant) / 8 * torch.exp2(e.double() - 7), mant / 8 * 2.0 ** -6)
        return (x.reshape(*raw.shape[:2], 128, 8, 16) * size[..., None]).reshape(x.shape)

    kc, vc, ic = s["caches"]
    out = torch.zeros(c["B"], c["G"] * c["Hkv"], D4, dtype=torch.float64, device="cuda")
    for b, L in enumerate(s["lens"].tolist()):
        if L == 0:
            continue
        n = (L + BLOCK - 1) // BLOCK
        pages = s["table"][b, :n].long()
        score = torch.empty(c["Hkv"], n, dtype=torch.float64, device="cuda")
        if n > TOPK:
            for a in range(0, n, 128):
                x = page(ic, pages[a:a + 128])
                score[:, a:a + 128] = torch.einsum("nhkd,hd->nhk", x, s["q_idx"][b].double()).amax(-1).T
        for h in range(c["Hkv"]):
            pick = list(range(n))
            if n > TOPK:
                first = list(range(min(c["n_init"], n - 1)))
                rest = score[h, len(first):n - 1].tolist()
                best = sorted(range(len(rest)), key=lambda i: (-rest[i], i))[:TOPK - 1 - len(first)]
                pick = sorted(first + [len(first) + i for i in best]) + [n - 1]
            at = pages[pick]
            K, V = page(kc[:, h:h + 1], at).reshape(-1, D4), page(vc[:, h:h + 1], at).reshape(-1, D4)
            keys = torch.cat([torch.arange(i * BLOCK, (i + 1) * BLOCK) for i in pick]).cuda() < L
            z = s["q"][b, h * c["G"]:(h + 1) * c["G"]].double() @ K[keys].T / math.sqrt(D4)
            out[b, h * c["G"]:(h + 1) * c["G"]] = torch.softmax(z, -1) @ V[keys]
    return out, None


if __name__ == "__main__":
    for case in listed() + [draw(random.Random(i)) for i in range(4)]:
        print(case, work(case))
