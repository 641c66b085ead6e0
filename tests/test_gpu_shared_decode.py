"""Append to 16-bit pages, attention over shared pages, beam selection and reordering of
rows on the GPU against fp64 definitions (oracle/shared_oracle.py, oracle/long_oracle.py).

Tolerances, derived before the first run.  2^-8 is the largest relative rounding of bf16,
2^-24 of fp32.
  * prologue: as in test_gpu_long_context.py, 2^-8 |y| + 2^-17 gain max|z|; v and what is not
    turned keep their bits.
  * logits: sums of 128 exact products in fp32 (tensor core, truncating): off by at most
    128 * 2^-23 sum|q k| = 2^-16 sum|q k|, times the scale.
  * weights p are rounded to bf16, their sum is not: |o error| <= (2^-8 + 2 e) max|v| + 2^-8 |o|
    with e the logits' error plus 2^-18 (exponentials, sums, the factors that join parts).
  * as a whole (2-norm): roundings of weights and output are independent and 0.42 2^-8 each
    on average: below 2^-8 together.
  * lse: e + 2^-22 |lse|.
  * log-sum-exp of logits: exponentials good to 2^-21 (2 units of ex2, the rounding of its
    argument, which stays below 2^5 where it matters): scores within 2^-20 + 2^-24 |score|, and
    the order is that of the 64-bit scores wherever these are 2^-19 apart or of one beam.
"""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import long_oracle as L
from oracle import shared_oracle as S

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
SCALE = 1.0 / math.sqrt(128)


@pytest.fixture(scope="module")
def m():
    import __graft_entry__ as ge
    ge.build()
    import msa_block_sparse_gb300 as mod
    return mod


def f64(t):
    return t.detach().cpu().double().numpy()


def bf16(x):
    return torch.tensor(np.asarray(x), dtype=torch.float32).to(torch.bfloat16).to(DEV)


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def within(got, want, tol, what):
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(got - want) - tol):.3e}"


# ------------------------------------------------------------------ append

APPEND = [
    # tokens of each row, tokens before, G, Hkv, R, layout, scaling, norms (q, k, qi, ki), index
    ([1], [0], 16, 1, 64, "half", "none", "qk", False),
    ([1] * 70, [5000 + 131 * i for i in range(70)], 16, 4, 64, "half", "yarn", "qkij", True),
    ([0, 5, 0, 300, 1], [3, 126, 9, 0, 127], 6, 2, 128, "interleaved", "linear", "qk", False),
    ([129, 7], [1000, 0], 1, 3, 32, "half", "ntk", "", True),
    ([33, 64, 2], [64, 0, 77], 3, 1, 16, "interleaved", "none", "qj", True),
    ([700, 900], [0, 130], 16, 4, 64, "half", "none", "ki", True),
    ([40], [131072 - 40], 2, 2, 96, "half", "yarn", "k", False),
    ([13, 13, 13], [0, 0, 0], 256, 1, 64, "half", "none", "qk", False),
    ([9, 4], [200, 3], 1, 200, 48, "interleaved", "none", "qk", False),
]


def append_case(n, before, G, Hkv, index, seed, extra_pages=2):
    rng = np.random.default_rng(seed)
    end = np.array(n) + np.array(before)
    maxp = max(S.blocks(e) for e in end) + 1 if max(end) < 131072 else 1024
    first = [b // 128 for b in before]                 # pages before the first new token are not needed
    need = [S.blocks(e) - f for e, f in zip(end, first)]
    P = sum(need) + extra_pages
    perm = rng.permutation(P)
    table, at = np.full((len(n), maxp), -1), 0
    for s in range(len(n)):
        for c in range(first[s], S.blocks(end[s])):
            table[s, c], at = perm[at], at + 1
    T = sum(n)
    x = {k: bf16(rng.standard_normal((T, h, 128))) for k, h in
         (("q", G * Hkv), ("k", Hkv), ("v", Hkv), ("q_idx", Hkv), ("k_idx", Hkv))}
    w = {k: bf16(0.1 * rng.standard_normal(128)) for k in "qkij"}
    caches = [torch.full((P, Hkv, 128, 128), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(3)]
    cu = np.concatenate([[0], np.cumsum(n)])
    pos = np.concatenate([b + np.arange(k) for b, k in zip(before, n)]).astype(np.int64)
    row = np.repeat(np.arange(len(n)), n)
    return x, w, caches, table, cu, end, pos, row


@pytest.mark.parametrize("case", APPEND, ids=lambda c: f"{len(c[0])}x{c[2]}x{c[3]}-{c[4]}{c[5][0]}-{c[7]}-{c[8]}")
def test_cache_append(m, case):
    n, before, G, Hkv, R, layout, scaling, norms, index = case
    x, w, (kc, vc, ic), table, cu, end, pos, row = append_case(n, before, G, Hkv, index, seed=len(n) + R)
    factor = 1.0 if scaling == "none" else 4.0
    rope = m.msa_rope(R, 1e7, layout=layout, scaling=scaling, factor=factor, orig_len=4096.0)
    f, gain = L.rope_freqs(R, 1e7, scaling, factor, 4096.0)
    wt = {k: w[k] if k in norms else None for k in "qkij"}
    kw = dict(w_q=wt["q"], w_k=wt["k"])
    if index:
        kw.update(q_idx=x["q_idx"], k_idx=x["k_idx"], kidx_cache=ic, w_qi=wt["i"], w_ki=wt["j"])
    q, qi = m.msa_cache_append(x["q"], x["k"], x["v"], kc, vc, i32(table), i32(cu), i32(end), rope, **kw)
    m.msa_check_status()
    page, slot = table[row, pos // 128], pos % 128

    def check(got, src, wk, what):
        z = f64(src)
        want = L.prologue(z, None if wk is None else f64(wk), pos, f, gain, layout)
        zmax = np.abs(L.prologue(z, None if wk is None else f64(wk), pos * 0, f, 1.0, layout)).max(-1, keepdims=True)
        within(got, want, 2.0 ** -8 * np.abs(want) + 2.0 ** -17 * gain * zmax, what)
    check(f64(q), x["q"], wt["q"], "q")
    check(f64(kc)[page, :, slot], x["k"], wt["k"], "k")
    assert torch.equal(vc[page, :, slot], x["v"])
    touched = np.zeros(kc.shape[:1] + (128,), bool)
    touched[page, slot] = True
    for c in (kc, vc) + ((ic,) if index else ()):
        assert (c.transpose(1, 2)[torch.tensor(~touched, device=DEV)] == 7.0).all()
    if index:
        check(f64(qi), x["q_idx"], wt["i"], "q_idx")
        check(f64(ic)[page, :, slot], x["k_idx"], wt["j"], "k_idx")
    else:
        assert qi is None and (ic == 7.0).all()
    # in place, and the same bits
    q2 = x["q"].clone()
    again = [torch.full_like(c, 7.0) for c in (kc, vc, ic)]
    if index:
        kw.update(kidx_cache=again[2])
    out, _ = m.msa_cache_append(q2, x["k"], x["v"], again[0], again[1], i32(table), i32(cu), i32(end), rope, q_out=q2,
                                **kw)
    assert out is q2 and torch.equal(q2, q) and torch.equal(again[0], kc) and torch.equal(again[1], vc)


def test_cache_append_is_the_prologue_and_the_decode_append(m):
    rng = np.random.default_rng(3)
    B, G, Hkv = 9, 16, 2
    lens = [1, 2, 128, 129, 300, 257, 256, 90, 1000]
    table = np.arange(9 * 8).reshape(9, 8)
    x = [bf16(rng.standard_normal((B, h, 128))) for h in (G * Hkv, Hkv, Hkv, Hkv, Hkv)]     # q q_idx k v k_idx
    w = [bf16(0.1 * rng.standard_normal(128)) for _ in range(4)]                             # q qi k ki
    a = [torch.zeros(72, Hkv, 128, 128, dtype=torch.bfloat16, device=DEV) for _ in range(3)]
    b = [torch.zeros_like(t) for t in a]
    q1, qi1 = m.msa_decode_append(*x, *w, *a, i32(table), i32(lens))
    q2, qi2 = m.msa_cache_append(x[0], x[2], x[3], b[0], b[1], i32(table), i32(np.arange(B + 1)), i32(lens),
                                 m.msa_rope(64, 1e7), w_q=w[0], w_k=w[2], q_idx=x[1], k_idx=x[4], kidx_cache=b[2],
                                 w_qi=w[1], w_ki=w[3])
    for s, t in zip([q1, qi1] + a, [q2, qi2] + b):       # another order of the same sums: one bf16 step at most
        d = f64(s) - f64(t)
        assert (np.abs(d) <= 2.0 ** -7 * np.abs(f64(s)) + 2.0 ** -17).all() and (d != 0).mean() < 0.01
    rope = m.msa_rope(64, 1e7)
    cu, end = i32([0, B]), i32([700 + B])
    pos = i32(700 + np.arange(B))
    got, _ = m.msa_cache_append(x[0], x[2], x[3], b[0], b[1], i32([list(range(8))]), cu, end, rope, w_q=w[0])
    assert torch.equal(got, m.msa_qk_norm_rope_ex(x[0], w[0], rope, positions=pos))
    m.msa_check_status()


def test_cache_append_padding_and_bad_places(m):
    """Rows of length 0 and tokens outside the sequences are left alone; bad places are reported."""
    rng = np.random.default_rng(4)
    T, G, Hkv, P = 30, 2, 2, 6
    x = [bf16(rng.standard_normal((T, h, 128))) for h in (G * Hkv, Hkv, Hkv)]
    for t in x:
        t[:3] = float("nan")
        t[25:] = float("nan")
    rope = m.msa_rope(64)
    cu = i32([3, 10, 15, 25])

    def run(table, lens):
        kc, vc = (torch.full((P, Hkv, 128, 128), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        q = torch.full_like(x[0], 7.0)
        m.msa_cache_append(*x, kc, vc, i32(table), cu, i32(lens), rope, q_out=q)
        return q, kc, vc
    q, kc, vc = run([[0, 1], [2, 3], [4, 5]], [7, 0, 130])
    m.msa_check_status()
    assert (q[:3] == 7).all() and (q[10:15] == 7).all() and (q[25:] == 7).all()
    assert torch.equal(vc[0, :, :7], x[2][3:10].transpose(0, 1)) and (vc[2:4] == 7).all() and (vc[0, :, 7:] == 7).all()
    assert torch.equal(vc[4, :, 120:], x[2][15:23].transpose(0, 1)) and torch.equal(vc[5, :, :2], x[2][23:25].transpose(0, 1))
    # lengths below the tokens, above the table, pages out of range: those tokens only
    for table, lens, bad in (([[0, 1], [2, 3], [4, 5]], [5, 9, 300], [0, 1] + list(range(16 - 3, 22))),
                             ([[-1, 1], [2, 6], [4, 5]], [7, 130, 20], list(range(7)) + [10, 11])):
        q, kc, vc = run(table, lens)
        with pytest.raises(m.MSAError, match="BOUNDS"):
            m.msa_check_status()
        touched = (q[3:25] != 7).flatten(1).any(1).cpu().numpy()
        start = np.array([lens[0] - 7] * 7 + [lens[1] - 5] * 5 + [lens[2] - 10] * 10)
        pos = start + np.concatenate([np.arange(7), np.arange(5), np.arange(10)])
        row = np.repeat([0, 1, 2], [7, 5, 10])
        ok = (pos >= 0) & (pos < 256)
        pg = np.where(ok, np.array(table)[row, np.clip(pos, 0, 255) // 128], -1)
        ok &= (pg >= 0) & (pg < P)
        assert np.array_equal(touched, ok) and not ok.all() and ok.any()
        assert (vc != 7).flatten(2).any(2).any(1).sum() == len(set(pg[ok]))
        for i in np.nonzero(ok)[0]:
            assert torch.equal(vc[pg[i], :, pos[i] % 128], x[2][3 + i])


# ------------------------------------------------------------------ attention

def tree_table(rng, groups, maxp=None, empties=()):
    """groups: nested (shared pages, children) with leaves (own tokens); a table whose rows share."""
    rows, at = [], [0]

    def fresh(n):
        at[0] += n
        return list(range(at[0] - n, at[0]))

    def walk(node, prefix):
        if isinstance(node, tuple):
            pages = prefix + fresh(node[0])
            for c in node[1]:
                walk(c, pages)
        else:
            rows.append((prefix + fresh(S.blocks(node)), len(prefix) * 128 + node))
    for g in groups:
        walk(g, [])
    for e in empties:
        rows.insert(e, ([], 0))
    maxp = maxp or max(1, max(len(r) for r, _ in rows))
    table = np.full((len(rows), maxp), -1)
    perm = rng.permutation(max(1, at[0]))
    for b, (r, _) in enumerate(rows):
        table[b, :len(r)] = perm[r] if r else []
    return table, np.array([n for _, n in rows]), max(1, at[0])


def widen(table, wide=True):
    """The table with columns behind it that no row uses: no longer one of the small calls, which
    take one launch and look for nothing that is shared."""
    return np.pad(table, ((0, 0), (0, 200)), constant_values=-1) if wide else table


def attend_check(m, G, Hkv, table, lens, P, **kw):
    """Against the definition, small calls in both forms."""
    if table.shape[1] <= 128:
        attend_check_one(m, G, Hkv, widen(table), lens, P, **kw)
    return attend_check_one(m, G, Hkv, table, lens, P, **kw)


def attend_check_one(m, G, Hkv, table, lens, P, seed=0, scale=SCALE, extra=0, q_gain=1.0, rows=None, garbage=True):
    rng = np.random.default_rng(seed)
    B, Hq = len(lens), G * Hkv
    q = bf16(q_gain * rng.standard_normal((B, Hq, 128)))
    g = torch.Generator(device=DEV).manual_seed(seed)
    kc, vc = (torch.randn(P + extra, Hkv, 128, 128, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))
    if garbage:                              # behind a row's end, and in pages of no row
        used = np.zeros((P + extra, 128), bool)
        for b, n in enumerate(lens):
            for c in range(S.blocks(n)):
                if 0 <= table[b, c] < P + extra:
                    used[table[b, c], :n - 128 * c] = True
        free = torch.tensor(~used, device=DEV)
        for c, v in ((kc, float("nan")), (vc, float("inf"))):
            c.transpose(1, 2)[free] = v
            c.transpose(1, 2)[free & (torch.arange(128, device=DEV) % 2 == 0)] = float("nan")
    tt, lt = i32(table), i32(lens)
    ws = torch.full((m.workspace_bytes("decode_shared", B, Hq, Hkv, table.shape[1]),), 255, dtype=torch.uint8, device=DEV)
    o, lse = m.msa_decode_shared(q, kc, vc, tt, lt, scale=scale, workspace=ws)
    pick = np.arange(B) if rows is None else np.array(rows)
    m.msa_check_status()
    t2 = table[pick]
    kn, vn = np.nan_to_num(f64(kc)), np.nan_to_num(f64(vc), posinf=0.0)
    want, wlse = S.attend(f64(q)[pick], kn, vn, t2, lens[pick], scale)
    go, gl = f64(o)[pick], f64(lse)[pick]
    for i, b in enumerate(pick):
        for h in range(Hkv):
            K, V = S.row_tokens(kn, table, b, h, lens[b]), S.row_tokens(vn, table, b, h, lens[b])
            sl = slice(h * G, (h + 1) * G)
            if len(K) == 0:
                assert (go[i, sl] == 0).all() and (gl[i, sl] == -np.inf).all()
                continue
            e = 2.0 ** -16 * scale * (np.abs(f64(q)[b, sl]) @ np.abs(K).T).max() + 2.0 ** -18
            within(go[i, sl], want[i, sl], (2.0 ** -8 + 2 * e) * np.abs(V).max() + 2.0 ** -8 * np.abs(want[i, sl]), f"o {b}")
            within(gl[i, sl], wlse[i, sl], e + 2.0 ** -22 * np.abs(wlse[i, sl]), f"lse {b}")
    if np.abs(want).max() > 0 and q_gain <= 1:
        assert np.linalg.norm(go - want) <= 2.0 ** -8 * np.linalg.norm(want)
    # the same bits again, into given outputs and another workspace
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    r = m.msa_decode_shared(q, kc, vc, tt, lt, scale=scale, out=o2, lse=lse2)
    assert r[0] is o2 and torch.equal(o2, o) and torch.equal(lse2, lse)
    o2 = q.clone()
    m.msa_decode_shared(o2, kc, vc, tt, lt, scale=scale, out=o2)
    assert torch.equal(o2, o)
    return q, kc, vc, tt, lt, o, lse


ROWS = [
    (16, 1, [1]), (16, 1, [127]), (16, 1, [128]), (16, 4, [129]), (1, 1, [300, 1, 128]), (3, 2, [64, 65, 63, 0, 191]),
    (12, 1, [1000, 0, 0, 2, 513]), (17, 1, [200, 330]), (40, 2, [129, 700]), (64, 1, [90, 257]), (128, 1, [130, 64, 1]),
    (100, 2, [5, 600]), (8, 8, [3000]), (2, 3, list(range(0, 400, 13))), (16, 2, [0, 0]),
]


@pytest.mark.parametrize("G,Hkv,lens", ROWS, ids=lambda v: str(v) if not isinstance(v, list) else f"{len(v)}rows{v[0]}")
def test_shared_attention_of_rows_apart(m, G, Hkv, lens):
    table, lens, P = tree_table(np.random.default_rng(G), [int(n) for n in lens])
    attend_check(m, G, Hkv, table, lens, P, seed=G + Hkv)


SMALL = [                                     # heads per KV head, KV heads, lengths, columns
    (16, 4, [4096, 1, 0, 2048], 32), (7, 1, [129], 2), (1, 8, [257, 256, 255], 3), (16, 1, [4096, 3969, 127], 32),
    (9, 2, [33, 31, 32, 65, 97, 128, 1, 64, 96, 127], 1), (8, 3, [512, 511, 385, 384], 4), (15, 1, [0, 0], 5),
    (3, 2, [640, 513, 1, 0], 5), (16, 19, [1024] * 4, 8), (16, 2, [1025, 1152, 2000, 900], 31), (10, 5, [1, 130], 9),
    (16, 4, [8192, 8065, 4096, 100], 64), (16, 2, [7000] * 19, 64), (16, 2, [16384, 129, 16000], 128), (4, 4, [2500] * 60, 20), (8, 2, [4700] * 60, 40), (5, 1, [3000] * 70, 32), (16, 64, [300], 3), (1, 1, [1], 1), (16, 1, [128] * 608, 1), (2, 1, [200] * 300, 2),
]


@pytest.mark.parametrize("G,Hkv,lens,cols", SMALL, ids=lambda v: str(v) if not isinstance(v, list) else f"{len(v)}rows{v[0]}")
def test_shared_attention_of_few_pages(m, G, Hkv, lens, cols):
    table, lens, P = tree_table(np.random.default_rng(cols), [int(n) for n in lens if n], maxp=cols,
                                empties=[i for i, n in enumerate(lens) if n == 0])
    attend_check(m, G, Hkv, table, lens, P, seed=G + cols, rows=list(range(min(len(lens), 12))))


TREES = [
    # G, Hkv, groups, empty rows in between
    (16, 1, [(1, [5, 5])], ()),
    (16, 2, [(3, [1, 128, 129, 300])], (1, 3)),
    (16, 1, [(2, [40] * 9)], ()),                          # two tiles: wide
    (16, 1, [(5, [7] * 16)], ()),                          # two full tiles
    (16, 2, [(5, [7] * 17)], (4,)),                        # a second pair of tiles with one row
    (6, 2, [(9, [(2, [30, 1]), (1, [200, 60, 5])]), (1, [(1, [(1, [1, 2])]), 300]), 77], (0, 5)),
    (1, 1, [(2, [3] * 150)], ()),                          # more rows than a tile
    (5, 3, [(1, [10] * 26 + [(4, [1, 2, 3])] * 2)], ()),
    (128, 1, [(3, [9, 9, 9])], ()),                        # a row is a tile
    (100, 1, [(2, [1, 1])], ()),
    (33, 1, [(2, [1] * 7)], ()),                           # three rows per tile
    (16, 1, [(40, [1] * 30), (33, [100, 30])], ()),
    (4, 1, [(20, [(j, [5, 6]) for j in range(1, 12)])], ()),
    (8, 1, [(300, [5] * 40)], ()),
]


@pytest.mark.parametrize("case", TREES, ids=lambda c: f"g{c[0]}x{c[1]}-{str(c[2])[:24]}")
def test_shared_attention_of_trees(m, case):
    G, Hkv, groups, empties = case
    table, lens, P = tree_table(np.random.default_rng(1), groups, empties=empties)
    attend_check(m, G, Hkv, table, lens, P, seed=G)


def test_shared_attention_of_a_staircase(m):
    """Every row shares one page more with the next than the one before did: deeper than the levels."""
    node = [130]
    for _ in range(20):
        node = [(1, [17] + node)]
    table, lens, P = tree_table(np.random.default_rng(2), node)
    attend_check(m, 16, 1, table, lens, P)
    attend_check(m, 4, 2, table[::-1].copy(), lens[::-1].copy(), P)


def test_shared_attention_of_random_tables(m):
    """Pages repeated within and between rows in any manner: still every row by itself."""
    rng = np.random.default_rng(5)
    for k in range(12):
        B, maxp, P = int(rng.integers(1, 40)), int(rng.integers(1, 9)), int(rng.integers(1, 6))
        lens = rng.integers(0, maxp * 128 + 1, B)
        lens[rng.random(B) < 0.3] = maxp * 128
        table = rng.integers(0, P, (B, maxp))
        if k % 2:                                         # rows alike but for a column
            table[:] = table[0]
            table[np.arange(B), rng.integers(0, maxp, B)] = rng.integers(0, P, B)
        attend_check(m, int(rng.choice([1, 6, 16, 20])), int(rng.integers(1, 4)), table, lens, P, seed=k, garbage=False)


def test_shared_attention_longest_row(m):
    table, lens, P = tree_table(np.random.default_rng(6), [(1000, [131072 - 128000, 3, 2000])], maxp=1024)
    assert lens[0] == 131072
    attend_check(m, 16, 1, table, lens, P)


def test_shared_attention_many_rows(m):
    table, lens, P = tree_table(np.random.default_rng(7), [(2, [int(n) for n in range(1, 1025)]), (1, [60] * 1024)])
    assert len(lens) == 2048
    attend_check(m, 1, 1, table, lens, P, rows=[0, 1, 511, 1023, 1024, 1025, 2047])
    with pytest.raises(m.MSAError, match="UNSUPPORTED"):
        m.msa_decode_shared(torch.zeros(2049, 1, 128, dtype=torch.bfloat16, device=DEV),
                            *[torch.zeros(1, 1, 128, 128, dtype=torch.bfloat16, device=DEV)] * 2,
                            torch.zeros(2049, 1, dtype=torch.int32, device=DEV),
                            torch.zeros(2049, dtype=torch.int32, device=DEV))


def test_shared_attention_beyond_4_gb(m):
    """Pages whose byte offsets pass 32 bits, in a cache of 5 GB."""
    P, Hkv = 40000, 4
    kc, vc = (torch.zeros(P, Hkv, 128, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    g = torch.Generator(device=DEV).manual_seed(8)
    pages = [39999, 33000, 12, 39000]
    for c in (kc, vc):
        c[pages] = torch.randn(4, Hkv, 128, 128, generator=g, device=DEV).to(torch.bfloat16)
    q = torch.randn(2, 16, 128, generator=g, device=DEV).to(torch.bfloat16)
    table, lens = np.array([[39999, 33000, 12], [39999, 33000, 39000]]), np.array([300, 384])
    o, lse = m.msa_decode_shared(q, kc, vc, i32(table), i32(lens))
    m.msa_check_status()
    small = {p: i for i, p in enumerate(pages)}
    t2 = np.vectorize(small.get)(table)
    want, wlse = S.attend(f64(q), f64(kc[pages]), f64(vc[pages]), t2, lens, SCALE)
    assert np.linalg.norm(f64(o) - want) <= 2.0 ** -8 * np.linalg.norm(want)
    within(f64(lse), wlse, 2.0 ** -10, "lse")


@pytest.mark.parametrize("wide", [False, True])
def test_shared_attention_bad_pages_and_lengths(m, wide):
    rng = np.random.default_rng(9)
    P, G, Hkv = 6, 4, 2
    q = bf16(rng.standard_normal((6, G * Hkv, 128)))
    kc, vc = (bf16(rng.standard_normal((P, Hkv, 128, 128))) for _ in range(2))
    good = np.array([[0, 1, 2, 3]] * 6)
    for table, lens in ((good, [-1, 513, 2 ** 31 - 1, 512, 0, 77]),
                        (np.array([[0, 9, 2, 3], [0, 9, 2, -4], [-1, 1, 2, 6], [6, 6, 6, 6], [0, 1, 2, 3], [5, -2 ** 31, 0, 0]]),
                         [512, 500, 400, 300, 512, 129])):
        lens, table = np.array(lens), widen(table, wide)
        o, lse = m.msa_decode_shared(q, kc, vc, i32(table), i32(lens))
        with pytest.raises(m.MSAError, match="BOUNDS"):
            m.msa_check_status()
        want, wlse = S.attend(f64(q), f64(kc), f64(vc), table, lens, SCALE)
        assert np.linalg.norm(f64(o) - want) <= 2.0 ** -8 * np.linalg.norm(want)
        fin = np.isfinite(wlse)
        assert np.array_equal(fin, np.isfinite(f64(lse))) and (f64(o)[~fin] == 0).all()
        within(f64(lse)[fin], wlse[fin], 2.0 ** -12, "lse")


@pytest.mark.parametrize("scale,q_gain", [(2.0 ** -64, 1.0), (2.0 ** -30, 1.0), (1.0, 30.0), (2.0 ** 20, 1.0), (2.0 ** 64, 1.0)])
@pytest.mark.parametrize("wide", [False, True])
def test_shared_attention_small_and_large_logits(m, scale, q_gain, wide):
    """Nothing but rounding where logits are all alike; one key where they are far apart."""
    table, lens, P = tree_table(np.random.default_rng(10), [(3, [100, 5] + [3] * 8), 129])
    table = widen(table, wide)
    if scale < 1:
        attend_check(m, 16, 1, table, lens, P, scale=scale)
        return
    q, kc, vc, tt, lt, o, lse = (None,) * 7
    rng = np.random.default_rng(11)
    q = bf16(q_gain * rng.standard_normal((len(lens), 16, 128)))
    kc, vc = (bf16(rng.standard_normal((P, 1, 128, 128))) for _ in range(2))
    o, lse = m.msa_decode_shared(q, kc, vc, i32(table), i32(lens), scale=scale)
    m.msa_check_status()
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
    z = [f64(q)[b] @ S.row_tokens(f64(kc), table, b, 0, lens[b]).T for b in range(len(lens))]
    for b in range(len(lens)):
        e = 2.0 ** -16 * (np.abs(f64(q)[b]) @ np.abs(S.row_tokens(f64(kc), table, b, 0, lens[b])).T).max()
        top2 = np.sort(z[b], 1)[:, -2:]
        sure = (top2[:, 1] - top2[:, 0] - 2 * e) * scale > 20          # the others weigh e^-20
        V = S.row_tokens(f64(vc), table, b, 0, lens[b])
        # p is 1 to 2^-21 and rounds to 1; o is v, off by e^-20 of the others and 2^-8
        want = V[z[b].argmax(1)]
        within(f64(o)[b][sure], want[sure], 2.0 ** -8 * np.abs(want[sure]) + 384 * math.exp(-20) * 8, "o")
        within(f64(lse)[b], z[b].max(1) * scale, (e + 2.0 ** -22 * np.abs(z[b]).max()) * scale + 7, "lse")


@pytest.mark.parametrize("wide", [False, True])
def test_shared_attention_products_of_minus_infinity(m, wide):
    """Keys whose products are -infinity weigh nothing, be it whole blocks, pages or parts of a row;
    a head that has no others counts as one without keys."""
    table, lens, P = tree_table(np.random.default_rng(13), [(5, [40] * 18), (3, [0, 300]), 700, 130], empties=())
    table = widen(table, wide)
    rng = np.random.default_rng(14)
    q = bf16(rng.standard_normal((len(lens), 16, 128)))
    q[:, :, 5] = 1.0
    kc, vc = (bf16(rng.standard_normal((P, 1, 128, 128))) for _ in range(2))
    for b, off in ((0, range(0, 3)), (18, range(1, 4)), (19, (0, 4)), (20, (0, 1, 2)), (21, (0, 1))):
        for c in off:
            if c < S.blocks(lens[b]):
                kc[table[b, c], 0, :, 5] = -math.inf
    kc[table[20, 3], 0, :64, 5] = -math.inf
    o, lse = m.msa_decode_shared(q, kc, vc, i32(table), i32(lens))
    m.msa_check_status()
    kn = np.where(np.isinf(f64(kc)), -1e30, f64(kc))
    want, wlse = S.attend(f64(q), kn, f64(vc), table, lens, SCALE)
    none = wlse < -1e20
    assert none.any() and not none.all()
    assert (f64(o)[none] == 0).all() and (f64(lse)[none] == -np.inf).all()
    assert np.linalg.norm(f64(o)[~none] - want[~none]) <= 2.0 ** -8 * np.linalg.norm(want[~none])
    within(f64(lse)[~none], wlse[~none], 2.0 ** -10, "lse")


@pytest.mark.parametrize("wide", [False, True])
def test_shared_attention_rows_and_heads_do_not_mix(m, wide):
    """A query row, or a row's own keys, that hold infinities or NaN change no other row."""
    table, lens, P = tree_table(np.random.default_rng(12), [(2, [40] * 12), 200])
    table = widen(table, wide)
    q, kc, vc, tt, lt, o, lse = attend_check(m, 16, 2, table, lens, P)
    bad = q.clone()
    bad[3, 5], bad[7, 20] = float("nan"), float("inf")
    kb, vb = kc.clone(), vc.clone()
    kb[table[5, 2], 1, 7], vb[table[5, 2], 1, 8] = float("nan"), float("inf")
    o2, lse2 = m.msa_decode_shared(bad, kb, vb, tt, lt)
    keep = torch.ones_like(lse, dtype=torch.bool)
    keep[3, 5] = keep[7, 20] = False
    keep[5, 16:] = False
    assert torch.equal(o2[keep], o[keep]) and torch.equal(lse2[keep], lse[keep])
    assert o2[3, 5].isnan().all() and o2[5, 16:].isnan().any()
    m.msa_check_status()


def test_shared_attention_equals_the_sparse_step_up_to_its_blocks(m):
    """Up to 16 blocks the block-sparse decode step attends to every key."""
    rng = np.random.default_rng(13)
    lens = [2048, 1, 700, 1999]
    table, lens, P = tree_table(rng, [int(n) for n in lens], maxp=16)
    q, qi = bf16(rng.standard_normal((4, 32, 128))), bf16(rng.standard_normal((4, 2, 128)))
    kc, vc, ic = (bf16(rng.standard_normal((P, 2, 128, 128))) for _ in range(3))
    a, _ = m.msa_decode_step(q, qi, kc, vc, ic, i32(table), i32(lens))
    b, _ = m.msa_decode_shared(q, kc, vc, i32(table), i32(lens))
    # both within 2^-8 of the definition in 2-norm
    assert np.linalg.norm(f64(a) - f64(b)) <= 2.0 ** -7 * np.linalg.norm(f64(b))
    m.msa_check_status()


# ------------------------------------------------------------------ beams

def beam_check(m, x, scores, W, K, finished=None, pad=0):
    so, po, to = m.msa_beam_select(x, scores, W, K, finished=finished, pad_token=pad)
    m.msa_check_status()
    fin = None if finished is None else finished.cpu().numpy()
    xs, ss = f64(x), f64(scores)
    every = S.beam_scores(xs, ss, fin, pad)
    ws, wp, wt = S.beam_select(xs, ss, W, K, fin, pad)
    gs, gp, gt = f64(so), po.cpu().numpy(), to.cpu().numpy()
    for n in range(len(ws)):
        live = ws[n] > -np.inf
        k = int(live.sum())
        assert (gp[n, k:] == -1).all() and (gt[n, k:] == -1).all() and (gs[n, k:] == -np.inf).all()
        assert (gp[n, :k] >= n * W).all() and (gp[n, :k] < (n + 1) * W).all()
        assert len(set(zip(gp[n, :k], gt[n, :k]))) == k
        mine = every[gp[n, :k], gt[n, :k]]
        lim = 2.0 ** -20 + 2.0 ** -23 * np.abs(ws[n, :k])
        within(gs[n, :k], mine, lim, "score")
        within(mine, ws[n, :k], 2 * lim, "order")
        same = (gp[n, :k] == wp[n, :k]) & (gt[n, :k] == wt[n, :k])
        # another choice only where scores of different beams are as near as their errors
        for i in np.nonzero(~same)[0]:
            near = np.abs(every[n * W:(n + 1) * W] - ws[n, i]) <= 2 * lim[i]
            assert near.any(1).sum() > 1, (n, i)
    return so, po, to


BEAMS = [
    # N, W, V, K, dtype, stride beyond V, masked, ended
    (1, 1, 1, 1, "f", 0, 0, 0), (1, 1, 64, 64, "b", 0, 0, 0), (1, 4, 32000, 4, "f", 0, 0, 0), (3, 5, 1009, 10, "f", 1, 0, 0.3),
    (2, 8, 4097, 16, "b", 3, 0.5, 0), (5, 2, 8193, 33, "b", 7, 0, 0.5), (1, 64, 700, 64, "f", 5, 0.9, 0), (2, 3, 100000, 64, "b", 0, 0, 0),
    (40, 4, 333, 5, "f", 11, 0.99, 0.2), (300, 2, 50, 3, "b", 0, 0, 0), (2, 2, 1 << 20, 8, "b", 1, 0, 0), (7, 3, 4, 12, "f", 0, 0.5, 0.5),
    (1, 64, 32000, 64, "b", 0, 0, 0.1), (4, 16, 50000, 16, "f", 1, 0, 0), (1, 32, 100000, 32, "b", 3, 0.5, 0),
]


@pytest.mark.parametrize("case", BEAMS, ids=lambda c: "-".join(map(str, c)))
def test_beam_select(m, case):
    N, W, V, K, dt, more, masked, ended = case
    g = torch.Generator(device=DEV).manual_seed(V + K)
    x = 3 * torch.randn(N * W, V + more, generator=g, device=DEV)
    x[torch.rand(x.shape, generator=g, device=DEV) < masked] = -math.inf
    x = x.to(torch.float32 if dt == "f" else torch.bfloat16)
    scores = -5 * torch.rand(N * W, generator=g, device=DEV)
    fin = torch.rand(N * W, generator=g, device=DEV) < ended if ended else None
    a = beam_check(m, x[:, :V], scores, W, K, fin, pad=V - 1)
    # rows elsewhere: the same choice from any alignment
    if more:
        y = torch.empty(N * W, V + more + 1, dtype=x.dtype, device=DEV)[:, 1:]
        y.copy_(x)
        b = m.msa_beam_select(y[:, :V], scores, W, K, finished=None if fin is None else fin.to(torch.uint8), pad_token=V - 1)
        assert all(torch.equal(p, q) for p, q in zip(a[1:], b[1:]))


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,W,K", [(5, 3, 7), (1000, 8, 16), (4097, 4, 64), (70001, 2, 20)])
def test_beam_select_values_alike_and_in_order(m, dt, V, W, K):
    """Ties, ascending and descending values, masks of the lowest value, NaN and infinities."""
    g = torch.Generator(device=DEV).manual_seed(V)
    scores = -torch.rand(2 * W, generator=g, device=DEV)
    low = torch.finfo(dt).min
    up = torch.arange(V, device=DEV).float().mul(1e-2).repeat(2 * W, 1).to(dt)
    few = torch.full((2 * W, V), low, device=DEV, dtype=dt)
    few[:, V // 2], few[:, V // 3] = 1.0, 0.5
    some = torch.randn(2 * W, V, generator=g, device=DEV).to(dt)
    some[0, V // 2], some[1, 0], some[1, V - 1] = math.nan, math.inf, math.inf
    some[2] = -math.inf
    for x in (torch.zeros(2 * W, V, device=DEV, dtype=dt), up, up.flip(1).contiguous(), few,
              torch.full_like(few, low), torch.full_like(few, -1e9), torch.full_like(few, -math.inf), some):
        beam_check(m, x, scores, W, K)
    scores[0], scores[W] = -math.inf, math.nan
    so, po, to = beam_check(m, some, torch.nan_to_num(scores, nan=-math.inf), W, min(K, (W - 1) * 2))
    again = m.msa_beam_select(some, scores, W, min(K, (W - 1) * 2))
    assert torch.equal(again[1], po) and torch.equal(again[2], to) and torch.equal(again[0], so)
    dead = m.msa_beam_select(some, torch.full_like(scores, -math.inf), W, K)
    assert (dead[0] == -math.inf).all() and (dead[1] == -1).all() and (dead[2] == -1).all()


@pytest.mark.parametrize("dt,V,more", [(torch.bfloat16, 300007, 1), (torch.float32, 160001, 3)])
def test_beam_select_many_rows_of_a_large_vocabulary(m, dt, V, more):
    """More rows than CTAs at a time: a CTA keeps one maximum for several tiles."""
    W, N = 4, 170
    g = torch.Generator(device=DEV).manual_seed(V)
    x = torch.empty(N * W, V + more, device=DEV, dtype=dt).normal_(0, 3, generator=g)[:, :V]
    scores = -torch.rand(N * W, generator=g, device=DEV)
    so, po, to = m.msa_beam_select(x, scores, W, 9)
    m.msa_check_status()
    for n in (0, 77, N - 1):
        s = slice(n * W, (n + 1) * W)
        ws, wp, wt = S.beam_select(f64(x[s]), f64(scores[s]), W, 9)
        within(f64(so[n:n + 1]), ws, 2.0 ** -20 + 2.0 ** -23 * np.abs(ws), "score")
        near = np.abs(np.diff(ws)).min() < 2.0 ** -18       # no choice between scores as near as their errors
        assert near or (np.array_equal(po[n:n + 1].cpu().numpy() - n * W, wp) and np.array_equal(to[n:n + 1].cpu().numpy(), wt))


def test_beam_select_best_values_side_by_side(m):
    """The K best of a row in one thread's hands, in one tile or one of each tile, and in falling order."""
    V, W, K = 262144, 2, 64
    base = torch.full((W, V), -20.0, device=DEV)
    vec, tile = 4, 256 * 16                                   # fp32: values of a load, values of a tile
    for where in ([8 * tile + 5 * vec + j + 1024 * u for u in range(4) for j in range(vec)] * 4,
                  [t * tile + 77 * vec + j for t in range(16) for j in range(vec)],
                  list(range(100000, 100064)), [V - 1 - i for i in range(64)]):
        for order in (1.0, -1.0, 0.0):
            x = base.clone()
            at = torch.tensor(sorted(set(where)), device=DEV)
            x[:, at] = 5 + order * 0.125 * torch.arange(len(at), device=DEV)
            beam_check(m, x, torch.tensor([-1.0, -1.0], device=DEV), W, K)


def test_beam_select_beams_alike(m):
    """The first step: all beams equal, the lowest takes every place."""
    x = torch.randn(1, 5000, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV).repeat(6, 1)
    so, po, to = m.msa_beam_select(x, torch.zeros(6, device=DEV), 3, 3)
    best = x[0].topk(1)[1]
    assert po.tolist() == [[0, 1, 2], [3, 4, 5]] and (to == best).all() and (so[:, 0] == so[:, 2]).all()
    first = torch.tensor([0.0, -math.inf, -math.inf] * 2, device=DEV)
    so, po, to = m.msa_beam_select(x, first, 3, 3)
    assert po.tolist() == [[0] * 3, [3] * 3] and torch.equal(to[0].long(), x[0].topk(3)[1])


def test_beam_select_scores_in_place(m):
    x = torch.randn(12, 3001, generator=torch.Generator(device=DEV).manual_seed(3), device=DEV)
    scores = -torch.arange(12.0, device=DEV) / 3
    want = m.msa_beam_select(x, scores, 4)
    got = m.msa_beam_select(x, scores, 4, scores_out=scores.view(3, 4))
    assert torch.equal(scores.view(3, 4), want[0]) and all(torch.equal(a, b) for a, b in zip(got, want))
    with pytest.raises(m.MSAError, match="overlaps"):
        m.msa_beam_select(x, scores, 4, n_out=2, scores_out=scores[:6].view(3, 2))


def test_beam_select_argument_checks(m):
    x, s = torch.zeros(4, 50, device=DEV), torch.zeros(4, device=DEV)
    for bad in (lambda: m.msa_beam_select(x.half(), s, 2), lambda: m.msa_beam_select(x, s, 3), lambda: m.msa_beam_select(x, s[:3], 2),
                lambda: m.msa_beam_select(x.t(), torch.zeros(50, device=DEV), 2), lambda: m.msa_beam_select(x, s.double(), 2),
                lambda: m.msa_beam_select(x, s, 2, 0), lambda: m.msa_beam_select(x, s, 0), lambda: m.msa_beam_select(x[0], s, 2),
                lambda: m.msa_beam_select(x, s, 2, finished=s), lambda: m.msa_beam_select(x[:1].expand(4, 50), s, 2),
                lambda: m.msa_beam_select(x, s, 2, parents=torch.zeros(2, 2, device=DEV)),
                lambda: m.msa_beam_select(x, s, 2, workspace=torch.zeros(8, dtype=torch.uint8, device=DEV)),
                lambda: m.msa_beam_select(x[:, ::2], s, 2), lambda: m.msa_beam_select(x, s.cpu(), 2)):
        with pytest.raises(ValueError):
            bad()
    for bad in (dict(n_out=65), dict(pad_token=50), dict(pad_token=-1)):
        with pytest.raises(m.MSAError):
            m.msa_beam_select(x, s, 2, **bad)


def test_decode_shared_and_append_argument_checks(m):
    bf = dict(dtype=torch.bfloat16, device=DEV)
    q, c = torch.zeros(2, 4, 128, **bf), torch.zeros(3, 2, 128, 128, **bf)
    table, lens = i32([[0, 1], [1, 2]]), i32([5, 130])
    for bad in (lambda: m.msa_decode_shared(q.float(), c, c, table, lens), lambda: m.msa_decode_shared(q, c, c[:2], table, lens),
                lambda: m.msa_decode_shared(q, c, c, table[:1], lens), lambda: m.msa_decode_shared(q, c, c, table, lens.long()),
                lambda: m.msa_decode_shared(q.transpose(0, 1), c, c, table, lens), lambda: m.msa_decode_shared(q, c[0], c, table, lens),
                lambda: m.msa_decode_shared(q, c, c, table, lens, lse=torch.zeros(2, 4, **bf)),
                lambda: m.msa_decode_shared(q, c, c, table, lens, workspace=torch.zeros(9, dtype=torch.uint8, device=DEV))):
        with pytest.raises(ValueError):
            bad()
    for kw in (dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan), dict(scale=2.0 ** 70)):
        with pytest.raises(m.MSAError):
            m.msa_decode_shared(q, c, c, table, lens, **kw)
    with pytest.raises(m.MSAError):
        m.msa_decode_shared(q[:, :3].contiguous(), c, c, table, lens)
    k, cu, rope, w = torch.zeros(2, 2, 128, **bf), i32([0, 1, 2]), m.msa_rope(64), torch.zeros(128, **bf)
    for bad in (dict(w_q=w.float()), dict(w_q=w[:64]), dict(q_idx=k), dict(q_idx=k, k_idx=k), dict(w_qi=w), dict(q_idx_out=k),
                dict(kidx_cache=c), dict(q_out=k)):
        with pytest.raises(ValueError):
            m.msa_cache_append(q, k, k, c, c, table, cu, lens, rope, **bad)
    with pytest.raises(ValueError):
        m.msa_cache_append(q, k, k[:1], c, c, table, cu, lens, rope)
    with pytest.raises(m.MSAError):
        m.msa_cache_append(q, k, k, c, c, table, cu, lens, m.msa_rope(256))
    m.msa_check_status()


# ------------------------------------------------------------------ rows in a new order

def reorder_state(rng, B, maxp, shared=0.3):
    lens = rng.integers(0, maxp * 128 + 1, B)
    lens[rng.random(B) < 0.2] = 0
    table, at = np.full((B, maxp), -1), 0
    for b in range(B):
        for j in range(S.blocks(lens[b])):
            if b and rng.random() < shared and table[b - 1, j] >= 0:
                table[b, j] = table[b - 1, j]
            else:
                table[b, j], at = at, at + 1
    P = at + 5
    perm = rng.permutation(P)
    table = np.where(table >= 0, perm[table], -1)
    ref = np.zeros(P, int)
    np.add.at(ref, table[table >= 0], 1)
    return table, lens, ref


@pytest.mark.parametrize("B,maxp", [(1, 1), (3, 2), (17, 5), (64, 256), (100, 300), (129, 513), (700, 97), (2, 1024), (65, 1024)])
def test_pages_reorder(m, B, maxp):
    rng = np.random.default_rng(B + maxp)
    table, lens, ref = reorder_state(rng, B, maxp)
    tt, lt, rt = i32(table), i32(lens), i32(ref)
    ws = torch.full((m.workspace_bytes("pages_reorder", B, maxp),), 255, dtype=torch.uint8, device=DEV)
    for k in range(4):
        parents = [np.arange(B), rng.integers(-1, B, B), rng.permutation(B), np.full(B, int(rng.integers(-1, B)))][(k + 1) % 4]
        table, lens, ref, kept = S.reorder(parents, table, lens, ref)
        got = m.msa_pages_reorder(i32(parents), tt, lt, rt, workspace=ws if k % 2 else None)
        m.msa_check_status()
        for a, b in ((tt, table), (lt, lens), (rt, ref), (got, kept)):
            assert np.array_equal(a.cpu().numpy(), b)


@pytest.mark.parametrize("B,maxp", [(12, 6), (300, 400)])
def test_pages_reorder_contradictions_are_reported(m, B, maxp):
    rng = np.random.default_rng(B)
    table, lens, ref = reorder_state(rng, B, maxp)
    lens = np.maximum(lens, 1) * (lens > 0) + (lens == 0) * 0
    ok = np.nonzero(lens > 0)[0]
    for bad_parent in (B, -2, 2 ** 31 - 1, -2 ** 31):
        parents = np.arange(B)
        parents[ok[0]], parents[ok[1]] = bad_parent, ok[2]
        tt, lt, rt = i32(table), i32(lens), i32(ref)
        got = m.msa_pages_reorder(i32(parents), tt, lt, rt)
        with pytest.raises(m.MSAError, match="BOUNDS"):
            m.msa_check_status()
        w = S.reorder(parents, table, lens, ref)
        assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip((tt, lt, rt, got), w)) and got[ok[0]] == -1
    # a parent with a length out of range; a row with such a length takes another's place
    l2 = lens.copy()
    l2[ok[3]] = maxp * 128 + 1
    parents = np.arange(B)
    parents[ok[0]], parents[ok[3]] = ok[3], ok[4]
    tt, lt, rt = i32(table), i32(l2), i32(ref)
    got = m.msa_pages_reorder(i32(parents), tt, lt, rt)
    with pytest.raises(m.MSAError, match="BOUNDS"):
        m.msa_check_status()
    w = S.reorder(parents, table, l2, ref)
    assert got[ok[0]] == -1 and got[ok[3]] == lens[ok[4]] and lt[ok[0]] == l2[ok[0]]
    assert np.array_equal(rt.cpu().numpy(), w[2])
    n = S.blocks(lens[ok[4]])
    assert np.array_equal(tt[ok[3], :n].cpu().numpy(), table[ok[4], :n])
    # counts below what the tables hold stay as they are, entries that are no pages are reported
    zero = i32(np.zeros_like(ref))
    tt, lt = i32(table), i32(lens)
    m.msa_pages_reorder(i32(np.full(B, -1)), tt, lt, zero)
    with pytest.raises(m.MSAError, match="BOUNDS"):
        m.msa_check_status()
    assert (zero == 0).all() and (lt == 0).all()
    t2 = table.copy()
    t2[ok[0], 0] = len(ref)
    tt, lt, rt = i32(t2), i32(lens), i32(ref)
    m.msa_pages_reorder(i32(np.where(np.arange(B) == ok[1], ok[0], np.arange(B))), tt, lt, rt)
    with pytest.raises(m.MSAError, match="BOUNDS"):
        m.msa_check_status()
    m.msa_check_status()


# ------------------------------------------------------------------ together

def loop_state(m, N, W, Hkv, G, prompt, maxp=6, V=97, seed=0):
    rng = np.random.default_rng(seed)
    B, P = N * W, N * (S.blocks(max(prompt)) + 2 * W * 3) + 8
    st = dict(table=i32(np.full((B, maxp), -1)), lens=i32(np.zeros(B)), ref=i32(np.zeros(P)),
              kc=torch.zeros(P, Hkv, 128, 128, dtype=torch.bfloat16, device=DEV),
              vc=torch.zeros(P, Hkv, 128, 128, dtype=torch.bfloat16, device=DEV), rope=m.msa_rope(64, 1e4),
              emb=bf16(rng.standard_normal((V, Hkv * G + 2 * Hkv, 128))), head=bf16(rng.standard_normal((V, Hkv * G * 128)) * 0.3),
              w=bf16(0.1 * rng.standard_normal(128)), V=V, rng=rng)
    return st


@pytest.mark.parametrize("maxp", [6, 200])
def test_beam_search_loop(m, maxp):
    """Prompts stored, forked to their beams and searched: every call against its definition, and
    at the end each row's pages hold the tokens that led to it."""
    N, W, Hkv, G, steps = 3, 4, 2, 3, 9
    prompt = [250, 129, 120]
    st = loop_state(m, N, W, Hkv, G, prompt, maxp=maxp)
    B, Hq, V = N * W, Hkv * G, st["V"]
    split = lambda e: (e[:, :Hq].contiguous(), e[:, Hq:Hq + Hkv].contiguous(), e[:, Hq + Hkv:].contiguous())   # noqa: E731
    toks = [st["rng"].integers(0, V, n) for n in prompt]
    caches = [st["kc"], st["vc"]]
    # prompts into the first row of each group
    add = np.zeros(B, int)
    add[::W] = prompt
    assert m.msa_pages_extend(i32(add), st["table"], st["lens"], st["ref"], caches).tolist() == [1] * B
    q, k, v = split(st["emb"][torch.tensor(np.concatenate(toks), device=DEV)])
    first = st["table"][::W].contiguous()
    m.msa_cache_append(q, k, v, *caches, first, i32(np.concatenate([[0], np.cumsum(prompt)])), i32(prompt), st["rope"],
                       w_q=st["w"], w_k=st["w"])
    src = np.repeat(np.arange(0, B, W), W - 1)
    dst = [b for b in range(B) if b % W]
    m.msa_pages_fork(i32(src), i32(dst), st["table"], st["lens"], st["ref"])
    scores = torch.tensor([0.0] + [-math.inf] * (W - 1), device=DEV).repeat(N)
    history = [list(toks[b // W]) for b in range(B)]
    last = torch.tensor([h[-1] for h in history], device=DEV)
    for step in range(steps):
        m.msa_pages_extend(i32(np.ones(B)), st["table"], st["lens"], st["ref"], caches)
        q, k, v = split(st["emb"][last])
        q, _ = m.msa_cache_append(q, k, v, *caches, st["table"], i32(np.arange(B + 1)), st["lens"], st["rope"],
                                  w_q=st["w"], w_k=st["w"])
        for h, t in zip(history, last.tolist()):
            h.append(t)
        o, lse = m.msa_decode_shared(q, *caches, st["table"], st["lens"])
        lens, table = st["lens"].cpu().numpy(), st["table"].cpu().numpy()
        want, wlse = S.attend(f64(q), f64(st["kc"]), f64(st["vc"]), table, lens, SCALE)
        assert np.linalg.norm(f64(o) - want) <= 2.0 ** -8 * np.linalg.norm(want)
        assert lens.tolist() == [len(h) for h in history]
        logits = (o.reshape(B, -1).float() @ st["head"].float().t())
        so, po, to = beam_check(m, logits, scores, W, W)
        t0, l0, r0 = table, lens, st["ref"].cpu().numpy()
        kept = m.msa_pages_reorder(po.view(-1), st["table"], st["lens"], st["ref"])
        m.msa_check_status()
        for a, b in zip((st["table"], st["lens"], st["ref"], kept), S.reorder(po.view(-1).cpu().numpy(), t0, l0, r0)):
            assert np.array_equal(a.cpu().numpy(), b)
        history = [list(history[p]) for p in po.view(-1).tolist()]
        scores, last = so.view(-1), to.view(-1).long()
    # v of a token is its embedding, unchanged: the pages tell the history
    lens, table, vc = st["lens"].cpu().numpy(), st["table"].cpu().numpy(), st["vc"].cpu()
    emb = st["emb"].cpu()[:, Hq + Hkv:]
    for b in range(B):
        rows = torch.cat([vc[table[b, c]].transpose(0, 1) for c in range(S.blocks(lens[b]))])[:lens[b]]
        assert torch.equal(rows, emb[torch.tensor(history[b])])


@pytest.mark.parametrize("maxp", [5, 200])
def test_captured_loop_follows_the_tables(m, maxp):
    """A step captured once and replayed while rows change places: what is shared is found out
    at each replay.  Beside it a second captured step on another stream with its own workspace."""
    N, W, Hkv, G = 2, 3, 1, 16
    table, lens, P = tree_table(np.random.default_rng(20), [(2, [100, 30, 64]), (1, [200, 128, 5])], maxp=maxp)
    B = len(lens)
    rng = np.random.default_rng(21)
    kc, vc = (bf16(rng.standard_normal((P + 30, Hkv, 128, 128))) for _ in range(2))
    ref = np.zeros(P + 30, int)
    np.add.at(ref, table[table >= 0], 1)
    side = [dict(table=i32(table), lens=i32(lens), ref=i32(ref), q=bf16(rng.standard_normal((B, G * Hkv, 128))),
                 x=torch.randn(B, 5001, device=DEV), scores=torch.zeros(B, device=DEV), stream=torch.cuda.Stream()) for _ in range(2)]

    def step(s):
        s["o"], s["lse"] = m.msa_decode_shared(s["q"], kc, vc, s["table"], s["lens"])
        s["so"], s["po"], s["to"] = m.msa_beam_select(s["x"], s["scores"], W)
        s["kept"] = m.msa_pages_reorder(s["po"].view(-1), s["table"], s["lens"], s["ref"])
    for s in side:
        with torch.cuda.stream(s["stream"]):
            step(s)
    torch.cuda.synchronize()
    for s in side:
        s["table"].copy_(i32(table)), s["lens"].copy_(i32(lens)), s["ref"].copy_(i32(ref))
        s["graph"] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(s["graph"], stream=s["stream"]):
            step(s)
    torch.cuda.synchronize()
    state = [(table, lens, ref)] * 2
    for k in range(5):
        for s in side:
            s["x"].normal_()
            s["q"].normal_()
        torch.cuda.synchronize()
        for s in side:
            with torch.cuda.stream(s["stream"]):
                s["graph"].replay()
        torch.cuda.synchronize()
        m.msa_check_status()
        for i, s in enumerate(side):
            t, n, r = state[i]
            want, wlse = S.attend(f64(s["q"]), f64(kc), f64(vc), t, n, SCALE)
            assert np.linalg.norm(f64(s["o"]) - want) <= 2.0 ** -8 * np.linalg.norm(want)
            ws, wp, wt = S.beam_select(f64(s["x"]), f64(s["scores"]), W, W)
            assert np.array_equal(s["po"].cpu().numpy(), wp) and np.array_equal(s["to"].cpu().numpy(), wt)
            t, n, r, kept = S.reorder(wp.ravel(), t, n, r)
            assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip((s["table"], s["lens"], s["ref"], s["kept"]), (t, n, r, kept)))
            state[i] = (t, n, r)


FIRST = """
import sys; sys.path.insert(0, {root!r})
import torch, msa_block_sparse_gb300 as m
d = 'cuda'; bf = dict(dtype=torch.bfloat16, device=d); i32 = dict(dtype=torch.int32, device=d)
B = 5
q, k = torch.randn(B, 32, 128, **bf), torch.randn(B, 2, 128, **bf)
kc, vc = torch.randn(9, 2, 128, 128, **bf), torch.randn(9, 2, 128, 128, **bf)
table = torch.tensor([[0, 1, 2 + b] + [-1] * {more} for b in range(B)], **i32)
lens, ref = torch.full((B,), 300, **i32), torch.tensor([5, 5, 1, 1, 1, 1, 1, 0, 0], **i32)
cu, x, s = torch.arange(B + 1, **i32), torch.randn(B, 999, device=d), torch.zeros(B, device=d)
rope, m_ = m.msa_rope(64), m
par = torch.tensor([1, 0, 2, 3, 4], **i32)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    a, _ = m.msa_cache_append(q, k, k, kc, vc, table, cu, lens, rope)
    o, lse = m.msa_decode_shared(a, kc, vc, table, lens)
    so, po, to = m.msa_beam_select(x, s, 5)
    kept = m.msa_pages_reorder(par, table, lens, ref)
g.replay(); torch.cuda.synchronize(); m.msa_check_status()
t0 = table.clone(); t0[0], t0[1] = table[1], table[0]
o2, lse2 = m.msa_decode_shared(a, kc, vc, t0, lens)
assert torch.equal(o2, o) and torch.equal(lse2, lse) and kept.tolist() == [300] * B
print('first ok')
"""


@pytest.mark.parametrize("more", [0, 200])
def test_first_calls_of_a_process_are_captured(m, more):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST.format(root=root, more=more)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "first ok" in r.stdout, r.stdout + r.stderr
