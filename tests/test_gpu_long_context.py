"""Long-context operators on the GPU against fp64 definitions (oracle/long_oracle.py).

Tolerances, derived before the first run.  u = 2^-24 is a rounding of fp32, 2^-8 the
largest relative rounding of bf16.
  * prologue: z = x r (1 + w) takes about 25 roundings on values below max|z| (a sum
    of up to 256 squares: 13; r: 3; products: 4), the turn two products of values below
    max|z| gain with angles good to 2^-24 of a turn (pi 2^-23 rad) and sincospi of a
    few u: below 2^-18 max|z| gain together, before the bf16 rounding.
  * dx = r (g - xh mean(g xh)): as above on terms below r max|g| (1 + max|xh|^2).
  * dw: a chain of at most 4096 additions, each term good to 2^-19 of its size:
    (4096 u + 2^-19) sum|dz xh| < 2^-11 sum|dz xh|; chains here are below 512
    additions, so 2^-14 sum|dz xh| holds.
  * 4-bit values are exact: equal bits.
  * attention, as a whole: roundings of the output (2^-8 at most each, 2^-9 on
    average) and of the weights (2^-11) are independent: below 2^-8 in 2-norm.
  * attention, value by value: logits are sums of 128 exact products in fp32 (tensor core, truncating:
    128 * 2^-22 of sum|q k| is far above it), scaled they are below ~16 in size: weights
    good to 2^-11 (fp16) + 16 * 2^-15; with the normaliser both count at most twice:
    |o error| <= (2^-10 + 2^-10) max|v| + 2^-8 |o|.
"""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import long_oracle as L

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
    bad = np.abs(got - want) > tol
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.max(np.abs(got - want) - tol):.3e}"


# ------------------------------------------------------------------ prologue

PRO = [
    # T, H, D, R, layout, scaling, norm, far
    (1, 1, 128, 64, "half", "none", True, 0),
    (33, 5, 128, 64, "half", "yarn", True, 0),
    (50, 12, 256, 256, "interleaved", "linear", True, 1000000),
    (129, 1, 256, 16, "half", "ntk", True, 0),
    (300, 2, 64, 64, "half", "none", True, 0),
    (7, 256, 64, 32, "interleaved", "yarn", True, 0),
    (70, 3, 256, 224, "half", "yarn", True, 2 ** 31 - 1),
    (41, 7, 128, 48, "interleaved", "none", False, 0),
    (17, 64, 128, 128, "half", "linear", False, 99),
    (2100, 17, 64, 16, "half", "yarn", True, 0),
]


def pro_case(T, H, D, R, layout, scaling, norm, far, seed=0):
    rng = np.random.default_rng(seed + T)
    x = f64(bf16(rng.standard_normal((T, H, D)) * 2.0 ** rng.integers(-3, 4, (T, H, 1))))
    dy = f64(bf16(rng.standard_normal((T, H, D))))
    w = f64(bf16(0.1 * rng.standard_normal(D))) if norm else None
    cu = np.sort(np.concatenate([[0, T], rng.integers(0, T + 1, 2)]))   # empty sequences too
    pos = rng.integers(0, far + 1, T) if far else L.positions_of(cu, T)
    if far:
        pos[0], pos[-1] = far, -5
    return x, dy, w, cu, pos


@pytest.mark.parametrize("case", PRO, ids=str)
def test_prologue_ex(m, case):
    T, H, D, R, layout, scaling, norm, far = case
    x, dy, w, cu, pos = pro_case(*case)
    f, gain = L.rope_freqs(R, 1e7, scaling, 4.0, 4096.0)
    rope = m.msa_rope(R, 1e7, layout=layout, scaling=scaling, factor=4.0, orig_len=4096.0)
    kw = dict(positions=i32(pos)) if far else dict(cu_seqlens=i32(cu))
    wt = None if w is None else bf16(w)
    y = m.msa_qk_norm_rope_ex(bf16(x), wt, rope, **kw)
    want = L.prologue(x, w, pos, f, gain, layout)
    zmax = np.abs(x if w is None else L.prologue(x, w, pos * 0, f, 1.0, layout)).max(-1, keepdims=True)
    within(f64(y), want, 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * 2 * gain * zmax, "y")
    # in place
    xt = bf16(x)
    assert m.msa_qk_norm_rope_ex(xt, wt, rope, out=xt, **kw) is xt and torch.equal(xt, y)

    dx, dw = m.msa_qk_norm_rope_bwd_ex(bf16(x), bf16(dy), wt, rope, **kw)
    wdx, wdw = L.prologue_bwd(x, dy, w, pos, f, gain, layout)
    if w is None:
        assert dw is None
        lim = 2.0 ** -18 * 2 * gain * np.abs(dy).max(-1, keepdims=True)
    else:
        r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6)
        dz = L.rotate(dy, pos, f, gain, layout, back=True)
        lim = 2.0 ** -18 * r * np.abs(dz * (1 + w)).max(-1, keepdims=True) * \
            (1 + np.abs(x * r).max(-1, keepdims=True) ** 2)
        within(f64(dw), wdw, 2.0 ** -14 * np.abs(dz * x * r).sum((0, 1)), "dw")
    within(f64(dx), wdx, 2.0 ** -8 * np.abs(wdx) + lim, "dx")
    # over dy, and the same bits again
    dyt = bf16(dy)
    dx2, dw2 = m.msa_qk_norm_rope_bwd_ex(bf16(x), dyt, wt, rope, dx=dyt, **kw)
    assert torch.equal(dx2, dx) and (dw is None or torch.equal(dw2, dw))
    m.msa_check_status()


@pytest.mark.parametrize("T,H,D,first,last", [(90, 3, 128, 7, 61), (40, 64, 64, 0, 1), (300, 5, 256, 128, 300),
                                              (12, 2, 128, 5, 5), (5000, 2, 64, 1, 4999)])
def test_prologue_ex_leaves_tokens_outside_the_sequences(m, T, H, D, first, last):
    rng = np.random.default_rng(T)
    x, dy = f64(bf16(rng.standard_normal((T, H, D)))), f64(bf16(rng.standard_normal((T, H, D))))
    w = bf16(0.1 * rng.standard_normal(D))
    cu = i32([first, (first + last) // 2, last])
    inside = slice(first, last)
    rope = m.msa_rope(32, 1e6)
    xt, dyt = bf16(x), bf16(dy)
    for t in (xt, dyt):                                  # what lies outside is not looked at
        t[:first] = float("nan")
        t[last:] = float("nan")
    y, dx = torch.full_like(xt, 7.0), torch.full_like(xt, 7.0)
    m.msa_qk_norm_rope_ex(xt, w, rope, cu_seqlens=cu, out=y)
    _, dw = m.msa_qk_norm_rope_bwd_ex(xt, dyt, w, rope, cu_seqlens=cu, dx=dx)
    pos = i32(np.concatenate([np.arange((first + last) // 2 - first), np.arange(last - (first + last) // 2)]))
    if last > first:
        xi, di = xt[inside].contiguous(), dyt[inside].contiguous()
        assert torch.equal(y[inside], m.msa_qk_norm_rope_ex(xi, w, rope, positions=pos))
        ref, dwi = m.msa_qk_norm_rope_bwd_ex(xi, di, w, rope, positions=pos)
        assert torch.equal(dx[inside], ref)
        # the same terms in another order: 2^-24 of their magnitudes per addition, 2^10 of them
        r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6)
        terms = (2 * np.abs(dy).max() * np.abs(x * r))[inside].sum((0, 1))
        within(f64(dw), f64(dwi), 2.0 ** -14 * terms, "dw")
    else:
        assert (dw == 0).all()
    for t in (y, dx):
        assert (t[:first] == 7.0).all() and (t[last:] == 7.0).all()
    m.msa_check_status()


def test_prologue_ex_is_the_fixed_prologue(m):
    """At the fixed layout it computes what msa_qk_norm_rope does (one bf16 step at most)."""
    rng = np.random.default_rng(5)
    x, w, cu = bf16(rng.standard_normal((500, 4, 128))), bf16(0.1 * rng.standard_normal(128)), i32([0, 123, 500])
    a = m.msa_qk_norm_rope(x, w, cu)
    b = m.msa_qk_norm_rope_ex(x, w, m.msa_rope(64, 1e7), cu_seqlens=cu)
    d = f64(a) - f64(b)
    assert (np.abs(d) <= 2.0 ** -7 * np.abs(f64(a)) + 2.0 ** -17).all() and (d != 0).mean() < 0.01


def test_prologue_gradient_against_differences(m):
    """Directional derivative of sum(y dy) by the fp64 definition at the kernel's inputs."""
    x, dy, w, cu, pos = pro_case(20, 2, 128, 64, "half", "yarn", True, 0, seed=9)
    f, gain = L.rope_freqs(64, 1e7, "yarn", 4.0, 4096.0)
    rope = m.msa_rope(64, 1e7, scaling="yarn", factor=4.0, orig_len=4096.0)
    dx, dw = m.msa_qk_norm_rope_bwd_ex(bf16(x), bf16(dy), bf16(w), rope, cu_seqlens=i32(cu))
    rng = np.random.default_rng(1)
    vx, vw, h = rng.standard_normal(x.shape), rng.standard_normal(128), 1e-5
    loss = lambda s: (L.prologue(x + s * vx, w + s * vw, pos, f, gain) * dy).sum()   # noqa: E731
    diff = (loss(h) - loss(-h)) / (2 * h)
    got = (f64(dx) * vx).sum() + (f64(dw) * vw).sum()
    # bf16 roundings of dx: independent, 2^-8 at most each
    lim = 2.0 ** -8 * np.abs(f64(dx) * vx).sum() + 1e-4 * abs(diff)
    assert abs(got - diff) <= lim


def test_prologue_ex_argument_checks(m):
    x, rope = torch.zeros(4, 2, 128, dtype=torch.bfloat16, device=DEV), m.msa_rope(64)
    pos = i32([0, 1, 2, 3])
    for bad in (dict(), dict(positions=pos, cu_seqlens=pos), dict(positions=pos[:3]),
                dict(positions=pos.long()), dict(cu_seqlens=pos[:1]), dict(positions=pos.cpu())):
        with pytest.raises(ValueError):
            m.msa_qk_norm_rope_ex(x, None, rope, **bad)
    for bx in (x.float(), x.transpose(0, 1), x[0]):
        with pytest.raises(ValueError):
            m.msa_qk_norm_rope_ex(bx, None, rope, positions=pos)
    with pytest.raises(ValueError):
        m.msa_qk_norm_rope_ex(x, None, "rope", positions=pos)
    with pytest.raises(m.MSAError):
        m.msa_qk_norm_rope_ex(x, None, m.msa_rope(256), positions=pos)


# ------------------------------------------------------------------ 4-bit cache

def layout_of(rng, ends, spare=2, max_pages=None):
    """Shuffled block table for rows that reach `ends` tokens; (table, pages)."""
    nb = -(-np.asarray(ends) // 128)
    P = int(nb.sum()) + spare
    perm = rng.permutation(P)
    t = np.full((len(ends), max_pages or max(1, int(nb.max()))), -1, np.int32)
    at = 0
    for b, n in enumerate(nb):
        t[b, :n] = perm[at:at + n]
        at += n
    return t, P


def spread(rng, *shape):
    """Values over many binades, zeros, ties and saturating blocks among them."""
    x = rng.standard_normal(shape) * 2.0 ** rng.integers(-9, 9, (*shape[:-1], 1))
    flat = x.reshape(-1, 16)
    flat[::7] = np.round(flat[::7] * 4) / 4            # ties of the codes
    flat[::11] = 0.0
    flat[5::13, 3] = 1e6
    flat[7::17, 0] = 6 * 2.0 ** -10
    return f64(bf16(x))


@pytest.mark.parametrize("lens,start,H,gains", [
    ((1,), 0, 1, (1, 1, 1)),
    ((128, 1, 0, 127), 0, 3, (1, 1, 1)),
    ((130, 37, 300), 777, 2, (0.25, 16.0, 2.0 ** -12)),
    ((40,), 127, 5, (1, 2.0 ** 20, 1)),
    ((600, 3), 5, 8, (1, 1, 1)),
])
def test_store_and_load(m, lens, start, H, gains):
    rng = np.random.default_rng(len(lens) + start)
    T, cu = int(np.sum(lens)), np.concatenate([[0], np.cumsum(lens)])
    first = np.full(len(lens), start)
    first[-1] += 3
    table, P = layout_of(rng, first + lens)
    x = [spread(rng, T + 2, H, 128) for _ in range(3)]     # two rows behind the last sequence
    x[1][0, 0, 5], x[2][T // 2, H - 1, 100] = np.nan, np.inf
    caches = [torch.full((P, H, 9216), 0x5A, dtype=torch.uint8, device=DEV) for _ in range(3)]
    kw = dict(start=i32(first), gains=gains)
    m.msa_cache4_store(*[bf16(a) for a in x], *caches, i32(table), i32(cu), **kw)
    got = m.msa_cache4_load(*caches, i32(table), i32(cu), T + 2, **kw,
                            **{n: torch.full((T + 2, H, 128), 7.0, dtype=torch.bfloat16, device=DEV)
                               for n in ("k", "v", "k_idx")})
    for a, c, y, g in zip(x, caches, got, gains):
        codes, scales = L.quantise(a[:T], g)
        assert np.array_equal(f64(y)[:T], L.held(codes, scales, g), equal_nan=True)
        assert (f64(y)[T:] == 7.0).all()                   # left as they were
        # the bytes: the format, and nothing else touched
        raw, seen = c.cpu().numpy(), np.full((P, H, 9216), 0x5A, np.uint8)
        byte = codes[..., 0::2] | (codes[..., 1::2] << 4)
        for s in range(len(lens)):
            for i in range(lens[s]):
                p, o = divmod(first[s] + i, 128)
                seen[table[s, p], :, 64 * o:64 * o + 64] = byte[cu[s] + i]
                seen[table[s, p], :, 8192 + 8 * o:8200 + 8 * o] = scales[cu[s] + i]
        assert np.array_equal(raw, seen)
    # one tensor alone
    only = m.msa_cache4_load(None, caches[1], None, i32(table), i32(cu), T, **kw)
    assert only[0] is None and only[2] is None
    assert np.array_equal(f64(only[1]), f64(got[1])[:T], equal_nan=True)
    m.msa_check_status()


def test_store_every_bf16_magnitude(m):
    """All finite bf16 magnitudes, alone with zeros and beside a larger value."""
    v = torch.arange(0x7F80, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    v = torch.cat([v, -v]).double().numpy()
    x = np.zeros((len(v), 8, 16))
    x[:, 0, 0] = v
    x[:, 1, :2] = np.stack([v, 2 * v], -1)
    x[:, 2, :2] = np.stack([v, 12 * v], -1)
    x[:, 3] = v[:, None] * np.linspace(0, 1, 16)
    x = np.nan_to_num(f64(bf16(np.clip(x, -3.3e38, 3.3e38).reshape(len(v), 1, 128))), posinf=3e38, neginf=-3e38)
    T = len(v)
    table, P = layout_of(np.random.default_rng(0), [T])
    cache = torch.zeros(P, 1, 9216, dtype=torch.uint8, device=DEV)
    m.msa_cache4_store(bf16(x), None, None, cache, None, None, i32(table), i32([0, T]))
    got = m.msa_cache4_load(cache, None, None, i32(table), i32([0, T]), T)[0]
    assert np.array_equal(f64(got), L.held(*L.quantise(x)))


def test_store_and_load_out_of_range(m):
    rng = np.random.default_rng(1)
    x = bf16(rng.standard_normal((300, 1, 128)))
    cache = torch.zeros(3, 1, 9216, dtype=torch.uint8, device=DEV)
    table = i32([[0, 3], [-1, 2]])                          # page 3 and -1 do not exist
    cu = i32([0, 200, 300])
    m.msa_cache4_store(x, None, None, cache, None, None, table, cu)
    with pytest.raises(m.MSAError, match="BOUNDS"):
        m.msa_check_status()
    y = m.msa_cache4_load(cache, None, None, table, cu, 300, start=i32([0, 200]))[0]
    with pytest.raises(m.MSAError, match="BOUNDS"):
        m.msa_check_status()
    want = np.zeros((300, 1, 128))
    want[:128] = L.held(*L.quantise(f64(x)[:128]))
    # row 1 starts at 200: its tokens 0 .. 55 are on page 2, which holds nothing yet
    assert np.array_equal(f64(y), want)
    m.msa_cache4_store(x, None, None, cache, None, None, table, cu, start=i32([-100, 300]))
    with pytest.raises(m.MSAError, match="BOUNDS"):
        m.msa_check_status()
    y = m.msa_cache4_load(cache, None, None, table, i32([0, 100, 100]), 100)[0]
    assert np.array_equal(f64(y), L.held(*L.quantise(f64(x)[100:200])))


def test_store_and_load_many_sequences(m):
    """More than 32 sequences (found by bisection), empty ones among them."""
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 9, 70)
    lens[[0, 5, 69]] = 0
    first = rng.integers(0, 300, 70)
    T, cu = int(lens.sum()), np.concatenate([[0], np.cumsum(lens)])
    table, P = layout_of(rng, first + lens)
    x = spread(rng, T, 2, 128)
    cache = torch.zeros(P, 2, 9216, dtype=torch.uint8, device=DEV)
    m.msa_cache4_store(None, bf16(x), None, None, cache, None, i32(table), i32(cu), start=i32(first))
    got = m.msa_cache4_load(None, cache, None, i32(table), i32(cu), T, start=i32(first))[1]
    want = L.held(*L.quantise(x))
    assert np.array_equal(f64(got), want)
    raw = L.slab_values(cache.cpu().numpy())
    for s in range(70):
        for i in range(lens[s]):
            p, o = divmod(first[s] + i, 128)
            assert np.array_equal(raw[table[s, p], :, o], want[cu[s] + i])
    m.msa_check_status()


def test_cache_beyond_4_gb(m):
    """Slabs whose offset in the cache passes 32 bits: store, load, decode and copies."""
    rng = np.random.default_rng(4)
    P, H, n = 120000, 4, 2300
    assert P * H * 9216 > 1 << 32
    nb = -(-n // 128)
    cache = torch.zeros(P, H, 9216, dtype=torch.uint8, device=DEV)
    pages = P - 1 - rng.permutation(2 * nb)
    table = pages[None, :nb].astype(np.int32)
    x = f64(bf16(rng.standard_normal((n, H, 128))))
    # one cache stands for all three: v and the index keys equal the keys
    m.msa_cache4_store(bf16(x), None, None, cache, None, None, i32(table), i32([0, n]))
    got = m.msa_cache4_load(cache, None, None, i32(table), i32([0, n]), n)[0]
    assert np.array_equal(f64(got), L.held(*L.quantise(x)))
    q, qi = (f64(bf16(rng.standard_normal((1, h, 128)))) for h in (4 * H, H))
    o, sel = m.msa_decode4_step(bf16(q), bf16(qi), cache, cache, cache, i32(table), i32([n]))
    slabs = cache[torch.tensor(pages[:nb].copy(), device=DEV)].cpu().numpy()
    local = np.arange(nb)[None]
    for h in range(H):
        want, gap = L.select(L.decode_scores(qi, slabs, local, 0, h, n))
        assert gap < 1e-5 or sel[0, h].tolist() == want
        ref = L.attend(q[0, 4 * h:4 * h + 4], slabs, slabs, local, 0, h, n, want, SCALE)
        within(f64(o)[0, 4 * h:4 * h + 4], ref, 2.0 ** -8 * np.abs(ref) + 2.0 ** -9 * 6, f"o[{h}]")
    m.msa_pages_copy(i32(pages[:nb]), i32(pages[nb:]), [cache])
    m.msa_pages_copy(i32(pages[:1]), i32([0]), [cache])
    t = torch.tensor(pages.copy(), device=DEV)
    assert torch.equal(cache[t[:nb]], cache[t[nb:]]) and torch.equal(cache[0], cache[t[0]])
    m.msa_check_status()


@pytest.mark.parametrize("G,H,R,layout,scaling", [
    (16, 4, 64, "half", "yarn"), (1, 1, 128, "interleaved", "none"), (3, 5, 16, "half", "ntk"),
    (12, 2, 96, "interleaved", "linear"),
])
def test_append(m, G, H, R, layout, scaling):
    rng = np.random.default_rng(G)
    lens = np.array([1, 128, 129, 0, 700, 77, 130000])
    B = len(lens)
    used = np.where(lens > 0, 1, 0)
    table = np.full((B, 1024), -1, np.int32)                # only the new token's page is there
    pages = rng.permutation(B + 1)
    for b in range(B):
        if used[b]:
            table[b, (lens[b] - 1) // 128] = pages[b]
    x = {n: rng.standard_normal((B, h, 128)) for n, h in (("q", G * H), ("q_idx", H), ("k", H), ("v", H),
                                                          ("k_idx", H))}
    x = {n: f64(bf16(a)) for n, a in x.items()}
    w = {n: f64(bf16(0.1 * rng.standard_normal(128))) for n in ("w_q", "w_qi", "w_k", "w_ki")}
    gains = (0.5, 4.0, 1.0)
    rope = m.msa_rope(R, 1e7, layout=layout, scaling=scaling, factor=4.0)
    f, gain = L.rope_freqs(R, 1e7, scaling, 4.0)
    caches = [torch.full((B + 1, H, 9216), 0x33, dtype=torch.uint8, device=DEV) for _ in range(3)]
    args = [bf16(x[n]) for n in ("q", "q_idx", "k", "v", "k_idx")] + \
        [bf16(w[n]) for n in ("w_q", "w_qi", "w_k", "w_ki")]
    out = [torch.full((B, h, 128), 9.0, dtype=torch.bfloat16, device=DEV) for h in (G * H, H)]
    m.msa_decode4_append(*args, *caches, i32(table), i32(lens), rope, gains=gains, q_out=out[0], q_idx_out=out[1])
    m.msa_check_status()
    pos, live = lens - 1, lens > 0
    pro = {n: L.prologue(x[n], w[wn], pos, f, gain, layout)
           for n, wn in (("q", "w_q"), ("q_idx", "w_qi"), ("k", "w_k"), ("k_idx", "w_ki"))}
    lim = lambda y: 2.0 ** -18 * 4 * gain * np.abs(y).max(-1, keepdims=True)      # noqa: E731
    for n, o in (("q", out[0]), ("q_idx", out[1])):
        within(f64(o)[live], pro[n][live], (2.0 ** -8 * np.abs(pro[n]) + lim(pro[n]))[live], n)
        assert (f64(o)[~live] == 9.0).all()                 # padding
    for n, c, g, ref in (("k", caches[0], gains[0], pro["k"]), ("v", caches[1], gains[1], x["v"]),
                         ("k_idx", caches[2], gains[2], pro["k_idx"])):
        raw = c.cpu().numpy()
        want = L.held(*L.quantise(L.bf16_round(ref), g), g)
        got = np.zeros_like(want)
        mask = np.ones(raw.shape, bool)
        for b in range(B):
            if live[b]:
                pg, o = table[b, pos[b] // 128], pos[b] % 128
                got[b] = L.slab_values(raw[pg], g)[:, o]
                mask[pg, :, 64 * o:64 * o + 64] = mask[pg, :, 8192 + 8 * o:8200 + 8 * o] = False
        assert (raw[mask] == 0x33).all()                    # nothing else was written
        same = got[live] == want[live]
        if n == "v":
            assert same.all()
        else:
            # a value next to a rounding border may go either way: rare, and then off by
            # one code of its block at most (2 scales) or one scale step (1/8)
            assert same.mean() > 0.995
            s = np.abs(want).reshape(B, H, 8, 16).max(-1, keepdims=True)
            off = (np.abs(got - want).reshape(B, H, 8, 16) / np.maximum(s, 1e-30))[live]
            assert off.max() <= 2 / 6 + 1 / 8


def test_append_out_of_range_leaves_the_row(m):
    rng = np.random.default_rng(0)
    B, H = 4, 2
    a = [bf16(rng.standard_normal((B, h, 128))) for h in (4, H, H, H, H)]
    w = [bf16(np.zeros(128))] * 4
    caches = [torch.zeros(3, H, 9216, dtype=torch.uint8, device=DEV) for _ in range(3)]
    q, qi = torch.full_like(a[0], 9.0), torch.full_like(a[1], 9.0)
    m.msa_decode4_append(*a, *w, *caches, i32([[0], [1], [5], [2]]), i32([-1, 129, 4, 3]), m.msa_rope(64),
                         q_out=q, q_idx_out=qi)
    with pytest.raises(m.MSAError, match="BOUNDS"):
        m.msa_check_status()
    assert (f64(q)[:3] == 9).all() and (f64(q)[3] != 9).any()
    assert all((c[:2] == 0).all() and (c[2] != 0).any() for c in caches)


# ------------------------------------------------------------------ decode step

def decode_case(rng, lens, G, H, spare=3, garbage=True, max_pages=None, gains=(1.0, 1.0)):
    table, P = layout_of(rng, lens, spare, max_pages)
    q = f64(bf16(rng.standard_normal((len(lens), G * H, 128))))
    qi = f64(bf16(rng.standard_normal((len(lens), H, 128))))
    slabs = []
    for n in range(3):
        x = rng.standard_normal((P, H, 128, 128))
        if n == 2:
            x += 0.5 * rng.standard_normal((P, H, 1, 128))
        g = (*gains, 1.0)[n]
        slabs.append(L.make_slab(f64(bf16(x * g)), g))
    if garbage:
        # slots behind the ends, and pages of no row, hold NaN scales
        for b, n in enumerate(lens):
            if n % 128:
                for s in slabs:
                    s[table[b, n // 128], :, 64 * (n % 128):8192] = 0xFF
                    s[table[b, n // 128], :, 8192 + 8 * (n % 128):] = 0x7F
        free = np.setdiff1d(np.arange(P), table[table >= 0])
        for s in slabs:
            s[free] = 0x7F
    return q, qi, slabs, table


def run_decode(m, q, qi, slabs, table, lens, **kw):
    c = [torch.tensor(s, device=DEV) for s in slabs]
    o, sel = m.msa_decode4_step(bf16(q), bf16(qi), *c, i32(table), i32(lens), **kw)
    return f64(o), sel.cpu().numpy()


def check_decode(m, lens, G, H, seed=0, n_init=0, gains=(1.0, 1.0), max_pages=None, scale=SCALE):
    rng = np.random.default_rng(seed)
    q, qi, slabs, table = decode_case(rng, lens, G, H, gains=gains, max_pages=max_pages)
    o, sel = run_decode(m, q, qi, slabs, table, lens, n_init=n_init, gains=(*gains, 1.0), scale=scale)
    m.msa_check_status()
    ties = 0
    refs = np.zeros_like(o)
    for b, n in enumerate(lens):
        for h in range(H):
            if n == 0:
                assert (sel[b, h] == -1).all() and (o[b] == 0).all()
                continue
            want, gap = L.select(L.decode_scores(qi, slabs[2], table, b, h, n), n_init)
            got = [x for x in sel[b, h] if x >= 0]
            assert (sel[b, h, len(got):] == -1).all()
            if got != want:
                # only where two scores around the border agree to fp32's accuracy
                assert gap < 1e-5 and len(got) == len(want) and got == sorted(set(got)) and got[-1] == want[-1]
                ties += 1
                want = got
            rows = slice(h * G, (h + 1) * G)
            ref = L.attend(q[b, rows], slabs[0], slabs[1], table, b, h, n, want, scale, *gains)
            refs[b, rows] = ref
            vmax = np.nanmax(np.abs(L.slab_values(slabs[1][table[b, want], h], gains[1])))
            within(o[b, rows], ref, 2.0 ** -8 * np.abs(ref) + 2.0 ** -9 * vmax, f"o[{b},{h}]")
    assert ties <= 1
    assert np.linalg.norm(o - refs) <= 2.0 ** -8 * np.linalg.norm(refs)


@pytest.mark.parametrize("lens,G,H,kw", [
    ((1,), 16, 1, {}),
    ((1, 127, 128, 129, 0, 2048, 2049), 16, 2, {}),
    ((2000, 0, 300), 1, 3, {}),
    ((5000, 2176, 4000, 2177), 6, 2, dict(n_init=3)),
    ((9000, 2305), 12, 1, dict(n_init=15)),
    ((3333, 17), 16, 4, dict(gains=(0.125, 64.0))),
    ((4100,), 7, 2, dict(max_pages=1024)),
    ((2500,) * 40, 2, 4, {}),
    ((2600, 100), 16, 1, dict(scale=2.0)),
    ((256, 512, 640, 300, 2048), 3, 1, {}),
    ((512,), 16, 1, {}),
    ((300, 2100, 0, 17, 2048, 640) * 4, 3, 3, {}),        # 72 rows, most of them short
    ((129, 5000, 1) * 13, 1, 1, {}),                      # 39 rows
    ((129, 2500, 1) * 27, 2, 1, dict(n_init=2)),          # 81 rows
    ((0, 0), 16, 2, {}),
    ((2100, 90) * 20, 15, 1, {}),                         # 40, 60, 100 and 160 rows of many heads
    ((700, 2300) * 15, 16, 2, {}),
    ((2200, 40) * 25, 16, 2, {}),
    ((100, 2100) * 40, 16, 2, dict(n_init=1)),
], ids=str)
def test_decode4(m, lens, G, H, kw):
    check_decode(m, lens, G, H, seed=len(lens), **kw)


def test_decode4_many_rows(m):
    """More rows than the score kernel counts at a time; some checked, all compared with the
    same rows alone."""
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 300, 1300)
    some = [0, 7, 500, 1023, 1024, 1025, 1299]
    lens[some] = [2200, 0, 2600, 2177, 3000, 130, 2049]
    q, qi, slabs, table = decode_case(rng, lens, 1, 1)
    o, sel = run_decode(m, q, qi, slabs, table, lens)
    m.msa_check_status()
    for b in some:
        if lens[b] == 0:
            assert (o[b] == 0).all() and (sel[b] == -1).all()
            continue
        want, gap = L.select(L.decode_scores(qi, slabs[2], table, b, 0, lens[b]))
        assert gap < 1e-5 or [x for x in sel[b, 0] if x >= 0] == want
        ref = L.attend(q[b], slabs[0], slabs[1], table, b, 0, lens[b], want, SCALE)
        within(o[b], ref, 2.0 ** -8 * np.abs(ref) + 2.0 ** -9 * 6, f"o[{b}]")
    pick = rng.permutation(1300)[:40]
    o2, sel2 = run_decode(m, q[pick], qi[pick], slabs, table[pick], lens[pick])
    assert np.array_equal(sel2, sel[pick])
    # other splits of a row's blocks over CTAs: other orders of the sums
    assert np.abs(o2 - o[pick]).max() <= 2.0 ** -7 * np.abs(o).max()


def test_decode4_beside_the_16_bit_step(m):
    """The same values held in 16 bits: msa_decode_step gives the same blocks and, within the
    two calls' roundings, the same output."""
    rng = np.random.default_rng(6)
    lens = (5000, 2049, 300, 4000)
    q, qi, slabs, table = decode_case(rng, lens, 16, 2, garbage=False)
    o, sel = run_decode(m, q, qi, slabs, table, lens)
    wide = [bf16(L.slab_values(s)) for s in slabs]
    ow, selw = m.msa_decode_step(bf16(q), bf16(qi), *wide, i32(table), i32(lens))
    m.msa_check_status()
    assert np.array_equal(selw.cpu().numpy(), sel)
    # its weights are rounded to bf16: 2^-8 each, independent
    assert np.linalg.norm(f64(ow) - o) <= 2.0 ** -7 * np.linalg.norm(o)


def test_decode4_longest(m):
    """1024 pages, the longest supported row, beside a short one."""
    check_decode(m, (131072, 70), 16, 1, seed=3)
    rng = np.random.default_rng(0)
    q, qi, slabs, table = decode_case(rng, (200,), 16, 1)
    with pytest.raises(m.MSAError, match="UNSUPPORTED"):
        run_decode(m, q, qi, slabs, np.pad(table, ((0, 0), (0, 1025)), constant_values=-1), (200,))


def test_decode4_exact_ties_go_to_the_lower_block(m):
    """Index pages copied from one another: equal scores, then a larger one."""
    rng = np.random.default_rng(7)
    q, qi, slabs, table = decode_case(rng, (128 * 40,), 16, 1, garbage=False)
    ki = slabs[2]
    base = ki[table[0, 0]].copy()
    double = base.copy()
    double[:, 8192:] = np.where(base[:, 8192:] > 0, base[:, 8192:] + 8, 0)   # scales times 2
    for c in range(39):
        ki[table[0, c]] = double if c in (5, 30, 38) else base
    _, sel = run_decode(m, q, qi, slabs, table, (128 * 40,))
    s = L.decode_scores(qi, ki, table, 0, 0, 128 * 40)
    assert s[5] == 2 * s[0]
    want, _ = L.select(s)
    assert sel[0, 0].tolist() == want


def test_decode4_bad_pages_and_lengths(m):
    rng = np.random.default_rng(8)
    lens = (3000, 129, 300, 400)
    q, qi, slabs, table = decode_case(rng, lens, 16, 2)
    table[0, 4], table[1, 0] = slabs[0].shape[0], -1
    bad = np.array([3000, 129, -3, 128 * table.shape[1] + 1])
    o, sel = run_decode(m, q, qi, slabs, table, bad)
    with pytest.raises(m.MSAError, match="BOUNDS"):
        m.msa_check_status()
    assert (sel[2:] == -1).all() and (o[2:] == 0).all()
    for b in (0, 1):
        for h in range(2):
            s = L.decode_scores(qi, slabs[2], table, b, h, bad[b])
            want, _ = L.select(s)
            assert [x for x in sel[b, h] if x >= 0] == want
            rows = slice(16 * h, 16 * h + 16)
            ref = L.attend(q[b, rows], slabs[0], slabs[1], table, b, h, bad[b], want, SCALE)
            within(o[b, rows], ref, 2.0 ** -8 * np.abs(ref) + 2.0 ** -9 * 6, "o")


def test_decode4_extreme_queries(m):
    """q over the whole range of bf16 (tiny rows, zero rows, huge rows) gives finite rows."""
    rng = np.random.default_rng(9)
    lens = (2500, 2500, 300)
    q, qi, slabs, table = decode_case(rng, lens, 16, 1, gains=(2.0 ** -60, 2.0 ** 30))
    q[0] = f64(bf16(q[0] * 1e-30))
    q[1, :8] = 0
    q[2] = f64(bf16(q[2] * 2.0 ** 55))
    qi[0] = f64(bf16(qi[0] * 1e-35))
    qi[1] = f64(bf16(qi[1] * 1e30))
    o, sel = run_decode(m, q, qi, slabs, table, lens, gains=(2.0 ** -60, 2.0 ** 30, 1.0))
    for b in range(3):
        want, gap = L.select(L.decode_scores(qi, slabs[2], table, b, 0, lens[b]))
        assert gap < 1e-5 or [x for x in sel[b, 0] if x >= 0] == want
        ref = L.attend(q[b], slabs[0], slabs[1], table, b, 0, lens[b], want, SCALE, 2.0 ** -60, 2.0 ** 30)
        within(o[b], ref, 2.0 ** -8 * np.abs(ref) + 2.0 ** -9 * 6 * 2.0 ** 30, f"o[{b}]")


def test_decode4_no_sel_out_and_argument_checks(m):
    import ctypes
    rng = np.random.default_rng(10)
    q, qi, slabs, table = decode_case(rng, (2500, 90), 16, 1)
    c = [torch.tensor(s, device=DEV) for s in slabs]
    qt, qit, tt, lt = bf16(q), bf16(qi), i32(table), i32((2500, 90))
    want, _ = m.msa_decode4_step(qt, qit, *c, tt, lt)
    ws = torch.empty(m.workspace_bytes("decode4_step", 2, 16, 1, table.shape[1]), dtype=torch.uint8, device=DEV)
    o = torch.empty_like(qt)
    p = lambda t: ctypes.c_void_p(t.data_ptr())    # noqa: E731
    rc = m.lib().msa_decode4_step(p(qt), p(qit), *[p(x) for x in c], p(tt), p(lt), 2, 16, 1, c[0].shape[0],
                                  table.shape[1], SCALE, 1.0, 1.0, 0, p(o), None, p(ws), ws.numel(),
                                  ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc == 0 and torch.equal(o, want)
    with pytest.raises(ValueError):
        m.msa_decode4_step(qt, qit, *c, tt, lt, workspace=ws[:16])
    with pytest.raises(ValueError):
        m.msa_decode4_step(qt, qit, c[0], c[1], c[2][:, :, :9000].contiguous(), tt, lt)
    with pytest.raises(ValueError):
        m.msa_decode4_step(qt, qit, *c, tt, lt.long())
    with pytest.raises(m.MSAError):
        m.msa_decode4_step(qt, qit, *c, tt, lt, gains=(3.0, 1.0, 1.0))


# ------------------------------------------------------------------ pages

class Gpu:
    """Tables and three caches of different page sizes on the GPU, beside the oracle's."""

    def __init__(self, m, B, P, maxp, seed=0):
        rng = np.random.default_rng(seed)
        self.m = m
        content = rng.integers(1, 1 << 30, P)
        self.o = L.Pages(np.full((B, maxp), -1), np.zeros(B, np.int64), np.zeros(P, np.int64), content)
        self.table, self.lens, self.ref = i32(self.o.table), i32(self.o.lens), i32(self.o.ref)
        c = i32(content)
        self.caches = [c[:, None].repeat(1, n).contiguous() for n in (4, 9216 // 4, 40000 // 4)]

    def check(self, what=""):
        self.m.msa_check_status()
        assert np.array_equal(self.lens.cpu().numpy(), self.o.lens), what
        assert np.array_equal(self.ref.cpu().numpy(), self.o.ref), what
        t = self.table.cpu().numpy()
        for b, n in enumerate(self.o.lens):
            k = L.Pages.blocks(n)
            assert np.array_equal(t[b, :k], self.o.table[b, :k]), what
        used = self.o.ref > 0
        for c in self.caches:
            x = c.cpu().numpy()
            assert (x[used] == self.o.content[used][:, None]).all(), what

    def fork(self, src, dst, keep=None):
        got = self.m.msa_pages_fork(i32(src), i32(dst), self.table, self.lens, self.ref,
                                    keep=None if keep is None else i32(keep))
        assert np.array_equal(got.cpu().numpy(), self.o.fork(src, dst, keep))

    def free(self, rows, keep=None):
        got = self.m.msa_pages_free(i32(rows), self.table, self.lens, self.ref,
                                    keep=None if keep is None else i32(keep))
        assert np.array_equal(got.cpu().numpy(), self.o.free(rows, keep))

    def extend(self, add):
        got = self.m.msa_pages_extend(i32(add), self.table, self.lens, self.ref, self.caches)
        assert np.array_equal(got.cpu().numpy(), self.o.extend(add))

    def compact(self):
        pm, n = self.m.msa_pages_compact(self.table, self.lens, self.ref, self.caches)
        wm, wn = self.o.compact()
        assert np.array_equal(pm.cpu().numpy(), wm) and n.item() == wn

    def write(self, b):
        """The row's last page gets new content (what an append does)."""
        pg = self.o.table[b, (self.o.lens[b] - 1) // 128]
        assert self.o.ref[pg] == 1
        self.o.content[pg] += 1
        for c in self.caches:
            c[pg] += 1


@pytest.mark.parametrize("B,P,maxp,seed", [(1, 1, 1, 0), (5, 12, 4, 1), (40, 100, 6, 2), (1500, 5000, 9, 3),
                                           (3, 4097, 1024, 4)])
def test_pages_random_operations(m, B, P, maxp, seed):
    g = Gpu(m, B, P, maxp, seed)
    rng = np.random.default_rng(seed)
    for step in range(25):
        kind = rng.integers(0, 5)
        if kind <= 1:
            add = rng.integers(0, rng.choice([2, 130, 128 * maxp + 2]), B) * (rng.random(B) < 0.6)
            before = g.o.lens.copy()
            g.extend(add)
            for b in np.nonzero(g.o.lens > before)[0][:20]:
                g.write(b)
        elif kind == 2:
            n = int(rng.integers(1, B + 2))
            src, dst = rng.integers(0, B, n), rng.integers(0, B, n)
            keep = None if rng.random() < 0.5 else (g.o.lens[src] * rng.random(n)).astype(int)
            g.fork(src, dst, keep)
        elif kind == 3:
            n = int(rng.integers(1, B + 2))
            rows = rng.integers(0, B, n)
            g.free(rows, None if rng.random() < 0.5 else rng.integers(0, 128 * maxp, n))
        else:
            g.compact()
        g.check(f"step {step}, kind {kind}")


def test_pages_pool_runs_out(m):
    g = Gpu(m, 6, 5, 8)
    g.extend([128, 128, 0, 300, 0, 128])        # 1 + 1 + 3 pages; the last row finds none
    assert g.o.lens.tolist() == [128, 128, 0, 300, 0, 0]
    g.check()
    g.extend([1, 0, 0, 0, 5, 0])                # nothing free
    g.check()
    g.free([1])
    g.fork([3], [1])
    g.extend([0, 1, 0, 1, 0, 0])                # one free page: the lower row copies, the other waits
    assert g.o.lens.tolist() == [128, 301, 0, 300, 0, 0]
    g.check()


def test_pages_contradictions_are_reported(m):
    B, P, maxp = 4, 6, 3

    def fresh():
        return (i32([[0, 1, -1], [2, 9, -1], [3, -1, -1], [-1, -1, -1]]), i32([200, 200, 50, 0]),
                i32([1, 1, 1, 0, 0, 0]))

    def bounds():
        with pytest.raises(m.MSAError, match="BOUNDS"):
            m.msa_check_status()

    t, n, r = fresh()
    out = m.msa_pages_fork(i32([7, 0, 1]), i32([3, -1, 3]), t, n, r)      # rows out of range; a page out of range
    bounds()
    assert out.tolist() == [-1, -1, 200] and r.tolist() == [1, 1, 2, 0, 0, 0]
    t, n, r = fresh()
    out = m.msa_pages_fork(i32([0]), i32([3]), t, n, r, keep=i32([500]))  # more than there is
    bounds()
    assert out.tolist() == [200] and n.tolist()[3] == 200
    t, n, r = fresh()
    out = m.msa_pages_free(i32([1, 2, -1]), t, n, r)                      # page 9; page 3 has no references
    bounds()
    assert out.tolist() == [200, 50, -1] and r.tolist() == [1, 1, 0, 0, 0, 0]
    t, n, r = fresh()
    out = m.msa_pages_extend(i32([-1, 1, 1, 1]), t, n, r, [])
    bounds()
    # row 1 ends on page 9, row 2 on a page that counts as free: both left; row 3 gets the first free page
    assert out.tolist() == [0, 0, 0, 1] and n.tolist() == [200, 200, 50, 1] and t[3, 0].item() == 3
    t, n, r = fresh()
    c = torch.arange(6, device=DEV, dtype=torch.int32)[:, None].repeat(1, 4).contiguous()
    pm, live = m.msa_pages_compact(t, n, r, [c])
    bounds()
    assert live.item() == 3 and pm.tolist() == [0, 1, 2, -1, -1, -1]
    m.msa_pages_copy(i32([0, 1, 2]), i32([3, 6, 2]), [c])
    bounds()
    assert c[:, 0].tolist() == [0, 1, 2, 0, 4, 5]


@pytest.mark.parametrize("words", [4, 4096, 4100, 40000])
def test_pages_copy(m, words):
    rng = np.random.default_rng(words)
    P = 600
    c = [torch.randint(-1000, 1000, (P, words), dtype=torch.int32, device=DEV),
         torch.randn(P, 2, 64, device=DEV).to(torch.bfloat16)]
    want = [x.clone() for x in c]
    perm = rng.permutation(P)
    src, dst = perm[:250], perm[250:500]
    m.msa_pages_copy(i32(src), i32(dst), c)
    for x, y in zip(c, want):
        y[torch.tensor(dst, device=DEV)] = y[torch.tensor(src, device=DEV)]
        assert torch.equal(x, y)
    m.msa_check_status()


# ------------------------------------------------------------------ together

def test_prefill_fork_decode_together(m):
    """A pack prefilled into the 4-bit cache, forked, and decoded for some steps with page
    upkeep, against the definitions on the held values; the pool is packed midway."""
    rng = np.random.default_rng(11)
    H, G, B, P, maxp = 2, 4, 6, 90, 24
    lens = np.array([2300, 128, 1])
    rope = m.msa_rope(64, 1e7, scaling="yarn", factor=4.0)
    w = {n: bf16(0.1 * rng.standard_normal(128)) for n in ("w_q", "w_qi", "w_k", "w_ki")}
    caches = [torch.zeros(P, H, 9216, dtype=torch.uint8, device=DEV) for _ in range(3)]
    table, cl, ref = i32(np.full((B, maxp), -1)), i32(np.zeros(B)), i32(np.zeros(P))
    assert m.msa_pages_extend(i32([*lens, 0, 0, 0]), table, cl, ref, caches).tolist() == [1] * 6
    T, cu = int(lens.sum()), i32(np.concatenate([[0], np.cumsum(lens)]))
    k, v, ki = (bf16(rng.standard_normal((T, H, 128))) for _ in range(3))
    k = m.msa_qk_norm_rope_ex(k, w["w_k"], rope, cu_seqlens=cu)
    ki = m.msa_qk_norm_rope_ex(ki, w["w_ki"], rope, cu_seqlens=cu)
    m.msa_cache4_store(k, v, ki, *caches, table[:3].contiguous(), cu)
    assert m.msa_pages_fork(i32([0, 0, 1]), i32([3, 4, 5]), table, cl, ref, keep=i32([2300, 1000, 128])).tolist() \
        == [2300, 1000, 128]
    for step in range(3):
        assert m.msa_pages_extend(i32(np.ones(B)), table, cl, ref, caches).tolist() == [1] * 6
        q, qi, kn, vn, kin = (bf16(rng.standard_normal((B, h, 128))) for h in (G * H, H, H, H, H))
        before = [c.clone() for c in caches]
        q, qi = m.msa_decode4_append(q, qi, kn, vn, kin, w["w_q"], w["w_qi"], w["w_k"], w["w_ki"], *caches, table,
                                     cl, rope)
        # every row wrote its own slot only: 64 + 8 bytes per row, head and cache at most
        for a, c in zip(before, caches):
            assert (a != c).sum().item() <= B * H * 72
        o, sel = m.msa_decode4_step(q, qi, *caches, table, cl)
        if step == 1:
            m.msa_pages_free(i32([2]), table, cl, ref)
            m.msa_pages_compact(table, cl, ref, caches)
            o2, sel2 = m.msa_decode4_step(q, qi, *caches, table, cl)
            keep = torch.tensor([0, 1, 3, 4, 5], device=DEV)
            assert torch.equal(o2[keep], o[keep]) and torch.equal(sel2[keep], sel[keep])
            assert (o2[2] == 0).all() and (sel2[2] == -1).all()
            m.msa_pages_fork(i32([4]), i32([2]), table, cl, ref)
            o, sel = m.msa_decode4_step(q, qi, *caches, table, cl)
        m.msa_check_status()
        tn, ln, slabs = table.cpu().numpy(), cl.cpu().numpy(), [c.cpu().numpy() for c in caches]
        for b in range(B):
            for h in range(H):
                want, gap = L.select(L.decode_scores(f64(qi), slabs[2], tn, b, h, ln[b]))
                got = [x for x in sel[b, h].tolist() if x >= 0]
                assert got == want or gap < 1e-5
                rows = slice(h * G, h * G + G)
                wo = L.attend(f64(q)[b, rows], slabs[0], slabs[1], tn, b, h, ln[b], got, SCALE)
                within(f64(o)[b, rows], wo, 2.0 ** -8 * np.abs(wo) + 2.0 ** -9 * 6, f"step {step} o[{b},{h}]")
    # forked rows hold their parents' tokens
    a = m.msa_cache4_load(*caches, table[:1].contiguous(), i32([0, 1000]), 1000)
    c = m.msa_cache4_load(*caches, table[4:5].contiguous(), i32([0, 1000]), 1000)
    assert all(torch.equal(x, y) for x, y in zip(a, c))


CAPTURE_FIRST = """
import torch, sys
import msa_block_sparse_gb300 as m
i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
bf = lambda *s: torch.randn(*s, device="cuda").bfloat16()
rope, B = m.msa_rope(64, 1e7), int(sys.argv[1])
caches = [torch.zeros(B * 20, 1, 9216, dtype=torch.uint8, device="cuda") for _ in range(3)]
table, lens, ref = i32([[-1] * 20] * B), i32([0] * B), i32([0] * (B * 20))
add, one, rows = i32([2300] * B), i32([1] * B), i32(list(range(B)))
w, x = bf(4, 128), [bf(B, h, 128) for h in (16, 1, 1, 1, 1)]
g, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
torch.cuda.synchronize()
with torch.cuda.graph(g, stream=st):
    m.msa_pages_extend(add, table, lens, ref, caches)
    m.msa_pages_extend(one, table, lens, ref, caches)
    q, qi = m.msa_decode4_append(*x, *w, *caches, table, lens, rope)
    o, sel = m.msa_decode4_step(q, qi, *caches, table, lens)
    m.msa_pages_free(rows, table, lens, ref)
for _ in range(2):
    g.replay()
torch.cuda.synchronize()
m.msa_check_status()
assert lens.tolist() == [0] * B and not ref.any() and bool(torch.isfinite(o.float()).all())
assert bool((sel[:, 0, -1] == 17).all())
"""


@pytest.mark.parametrize("B", [2, 30, 60, 100, 200])     # each choice of CTAs per row
def test_first_calls_of_a_process_are_captured(m, B):
    r = subprocess.run([sys.executable, "-c", CAPTURE_FIRST, str(B)], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, r.stderr[-2000:]


def test_captured_steps_and_streams(m):
    """Two captured decode loops with their own workspaces replay with new contents, also
    side by side on two streams, and equal the eager calls."""
    rng = np.random.default_rng(12)
    H, G, B, P, maxp = 2, 16, 3, 80, 30
    w = [bf16(0.1 * rng.standard_normal(128)) for _ in range(4)]
    rope = m.msa_rope(64, 1e7)
    sides = []
    for n in range(2):
        lens = rng.integers(2100, 2600, B)
        s = dict(cl=i32(np.zeros(B)), table=i32(np.full((B, maxp), -1)), ref=i32(np.zeros(P)), add=i32(lens),
                 x=[bf16(rng.standard_normal((B, h, 128))) for h in (G * H, H, H, H, H)],
                 caches=[torch.tensor(L.make_slab(rng.standard_normal((P, H, 128, 128))), device=DEV)
                         for _ in range(3)],
                 ws=torch.empty(m.workspace_bytes("decode4_step", B, G * H, H, maxp), dtype=torch.uint8, device=DEV),
                 pws=torch.empty(m.workspace_bytes("pages_extend", B, P), dtype=torch.uint8, device=DEV),
                 done=i32(np.zeros(B)), one=i32(np.ones(B)), stream=torch.cuda.Stream())
        m.msa_pages_extend(s["add"], s["table"], s["cl"], s["ref"], s["caches"])

        def step(s=s):
            m.msa_pages_extend(s["one"], s["table"], s["cl"], s["ref"], s["caches"], done=s["done"],
                               workspace=s["pws"])
            q, qi = m.msa_decode4_append(*s["x"], *w, *s["caches"], s["table"], s["cl"], rope)
            return m.msa_decode4_step(q, qi, *s["caches"], s["table"], s["cl"], workspace=s["ws"])

        s["step"] = step
        sides.append(s)
    names = ("cl", "table", "ref")
    torch.cuda.synchronize()
    saved = [({n: s[n].clone() for n in names}, [c.clone() for c in s["caches"]]) for s in sides]

    def restore():
        for s, (a, c) in zip(sides, saved):
            for n in names:
                s[n].copy_(a[n])
            for x, y in zip(s["caches"], c):
                x.copy_(y)
        torch.cuda.synchronize()

    eager = [[tuple(t.clone() for t in s["step"]()) for _ in range(3)] for s in sides]
    restore()
    graphs = []
    for s in sides:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s["stream"]):
            s["out"] = s["step"]()
        graphs.append(g)
    restore()
    for k in range(3):
        for s, g in zip(sides, graphs):
            with torch.cuda.stream(s["stream"]):
                g.replay()
        torch.cuda.synchronize()
        for s, want in zip(sides, eager):
            assert torch.equal(s["out"][0], want[k][0]) and torch.equal(s["out"][1], want[k][1])
    m.msa_check_status()
