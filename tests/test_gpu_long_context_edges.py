"""Long-context operators on the GPU where their arithmetic or their order of steps could
go wrong: values that are not finite or far from 1, rows that grow by many pages.
Helpers, definitions and tolerances are those of test_gpu_long_context.py."""
import math

import numpy as np
import pytest
import torch

from oracle import long_oracle as L
from tests import test_gpu_long_context as base

pytestmark = pytest.mark.gpu
m = base.m


# ------------------------------------------------------------------ pages

@pytest.mark.parametrize("B,maxp,seed", [(1, 1024, 0), (32, 200, 1), (33, 70, 2), (200, 33, 3)])
def test_extend_by_more_pages_than_lanes(m, B, maxp, seed):
    """Each row is served by a warp: pages of every trip of its lanes are placed by the length
    before the call, with and without a copy of a shared last page."""
    g = base.Gpu(m, B + 1, (B + 1) * maxp + 8, maxp, seed)
    rng = np.random.default_rng(seed)
    g.extend(np.concatenate([rng.integers(1, 200, B), [0]]))       # partly filled last pages
    g.fork([0], [B])                                               # row 0 and the last share theirs
    g.check("forked")
    g.extend([128 * maxp - n if b % 2 == 0 else 1 for b, n in enumerate(g.o.lens)])
    assert (g.o.lens[::2] == 128 * maxp).all()
    g.check("filled")
    g.extend([128 * maxp - n for n in g.o.lens])
    assert (g.o.lens == 128 * maxp).all()
    g.check("all filled")


# ------------------------------------------------------------------ comparisons that fail on NaN

def strict(got, want, tol, what):
    ok = np.abs(got - want) <= tol
    assert ok.all(), f"{what}: {(~ok).sum()} of {ok.size} off, {np.isnan(got).sum()} NaN"


def cases_of(test):
    """The parameters that a test of the other file runs with."""
    return [mark.args[1] for mark in test.pytestmark if mark.name == "parametrize"][0]


@pytest.fixture
def nan_fails(monkeypatch):
    """The other file's comparisons are of the form `error > tolerance`, which no NaN meets."""
    monkeypatch.setattr(base, "within", strict)


@pytest.mark.parametrize("case", base.PRO, ids=str)
def test_prologue_ex_without_nan(m, nan_fails, case):
    base.test_prologue_ex(m, case)


@pytest.mark.parametrize("case", cases_of(base.test_prologue_ex_leaves_tokens_outside_the_sequences), ids=str)
def test_tokens_outside_without_nan(m, nan_fails, case):
    base.test_prologue_ex_leaves_tokens_outside_the_sequences(m, *case)


@pytest.mark.parametrize("case", cases_of(base.test_append), ids=str)
def test_append_without_nan(m, nan_fails, case):
    base.test_append(m, *case)


@pytest.mark.parametrize("test", [base.test_decode4_extreme_queries, base.test_decode4_bad_pages_and_lengths,
                                  base.test_decode4_many_rows, base.test_cache_beyond_4_gb,
                                  base.test_prefill_fork_decode_together], ids=lambda f: f.__name__)
def test_decode4_without_nan(m, nan_fails, test):
    test(m)
    m.msa_check_status()


# ------------------------------------------------------------------ decode: logits near 0 and far from it

def check_attention(m, lens, q, qi, slabs, table, scale, gains, ref_of=None):
    o, sel = base.run_decode(m, q, qi, slabs, table, lens, scale=scale, gains=(*gains, 1.0))
    m.msa_check_status()
    assert np.isfinite(o).all()
    G = q.shape[1] // qi.shape[1]
    for b, n in enumerate(lens):
        for h in range(qi.shape[1]):
            picked = [x for x in sel[b, h] if x >= 0]
            want, gap = L.select(L.decode_scores(qi, slabs[2], table, b, h, n))
            assert gap < 1e-5 or picked == want
            rows = slice(h * G, (h + 1) * G)
            ref = L.attend(q[b, rows], slabs[0], slabs[1], table, b, h, n, picked, scale, *gains)
            vmax = np.nanmax(np.abs(L.slab_values(slabs[1][table[b, picked], h], gains[1])))
            strict(o[b, rows], ref, 2.0 ** -8 * np.abs(ref) + 2.0 ** -9 * vmax, f"o[{b},{h}]")


@pytest.mark.parametrize("G,H", [(16, 1), (3, 2)])
@pytest.mark.parametrize("scale,k_gain", [
    (base.SCALE, 1.0), (base.SCALE, 2.0 ** -28), (base.SCALE, 2.0 ** -64), (1e-30, 1.0), (1e-38, 1.0),
    (1e-38, 2.0 ** -64), (1e18, 2.0 ** -64), (1e-30, 2.0 ** 64)])
def test_decode4_small_logits(m, scale, k_gain, G, H):
    """Zero, tiny and ordinary heads at every accepted scale of the logits, in rows whose own block
    is partly filled: masked keys have no weight however flat the softmax is."""
    rng = np.random.default_rng(20)
    lens = (2500, 68, 1, 300, 129, 4000)
    q, qi, slabs, table = base.decode_case(rng, lens, G, H, gains=(k_gain, 1.0))
    q[:, 0] = 0.0
    q[:3, 1] = base.f64(base.bf16(q[:3, 1] * 1e-30))
    q[1:, 2] = base.f64(base.bf16(q[1:, 2] * 2.0 ** -126))     # down to subnormal values
    check_attention(m, lens, q, qi, slabs, table, scale, (k_gain, 1.0))


@pytest.mark.parametrize("up,k_gain", [(20, 1.0), (24, 1.0), (31, 1.0), (40, 1.0), (120, 1.0), (60, 2.0 ** 64),
                                       (120, 2.0 ** 64)])
def test_decode4_large_logits(m, up, k_gain):
    """Heads whose logits reach 2^20 to 2^184: the softmax is finite, and all on the largest one."""
    rng = np.random.default_rng(21)
    lens = (2500, 68, 300, 4000)
    q, qi, slabs, table = base.decode_case(rng, lens, 16, 1, gains=(k_gain, 1.0))
    # the two largest logits of a head lie far enough apart for the sums of 128 products that
    # decide between them (2^-18 of the products' magnitudes, far above fp32's rounding of them)
    for b, n in enumerate(lens):
        sel, _ = L.select(L.decode_scores(qi, slabs[2], table, b, 0, n))
        K = np.concatenate([L.slab_values(slabs[0][table[b, c], 0])[:min(128, n - 128 * c)] for c in sel])
        z = q[b] @ K.T
        top = np.sort(z, -1)
        assert ((top[:, -1] - top[:, -2]) > 2.0 ** -18 * (np.abs(q[b]) @ np.abs(K).T).max(-1)).all()
        assert ((top[:, -1] - top[:, -2]) * base.SCALE * 2.0 ** up > 200).all()
    q = q * 2.0 ** up
    check_attention(m, lens, q, qi, slabs, table, base.SCALE, (k_gain, 1.0))


def test_decode4_heads_do_not_mix(m):
    """A head whose query is not finite leaves the row's other heads as they are."""
    rng = np.random.default_rng(22)
    lens = (2500, 70)
    q, qi, slabs, table = base.decode_case(rng, lens, 16, 1)
    o, sel = base.run_decode(m, q, qi, slabs, table, lens)
    bad = q.copy()
    bad[0, 3, 5], bad[1, 9, 100] = np.nan, np.inf
    ob, selb = base.run_decode(m, bad, qi, slabs, table, lens)
    m.msa_check_status()
    keep = np.ones((2, 16), bool)
    keep[0, 3] = keep[1, 9] = False
    assert np.array_equal(sel, selb) and np.array_equal(o[keep], ob[keep]) and np.isfinite(o).all()
    assert not np.isfinite(ob[0, 3]).any()


def test_decode4_repeats_itself(m):
    """The same call gives the same bits."""
    rng = np.random.default_rng(23)
    for lens in ((2500, 70), (3000, 2200, 129) * 30):
        args = base.decode_case(rng, lens, 16, 1)
        first = base.run_decode(m, *args, lens)
        for _ in range(5):
            o, sel = base.run_decode(m, *args, lens)
            assert np.array_equal(o, first[0]) and np.array_equal(sel, first[1])


# ------------------------------------------------------------------ rotation: channels that are not rotated

ROT = [(9, 3, 128, 64, "half"), (33, 2, 128, 32, "interleaved"), (5, 7, 256, 224, "half"), (40, 5, 64, 16, "half"),
       (12, 4, 256, 16, "interleaved"), (6, 1, 128, 112, "interleaved")]


def spoil(x, R, rng):
    """A copy with an infinity, a NaN, a -0 and a huge value in channels behind the rotated ones of
    different rows, and where they are."""
    bad = x.clone()
    T, H, D = x.shape
    at = []
    for i, v in enumerate((math.inf, -math.inf, math.nan, -0.0, 3e38)):
        t, h, c = i % T, int(rng.integers(H)), int(rng.integers(R, D))
        bad[t, h, c] = v
        at.append((t, h, c))
    return bad, at


@pytest.mark.parametrize("T,H,D,R,layout", ROT)
def test_rotation_alone_passes_other_channels_through(m, T, H, D, R, layout):
    rng = np.random.default_rng(30)
    x = base.bf16(rng.standard_normal((T, H, D)))
    rope = m.msa_rope(R, 1e6, layout=layout, scaling="yarn", factor=4.0)
    pos = base.i32(rng.integers(0, 100000, T))
    bad, _ = spoil(x, R, rng)

    def turn(a, back, out=None):
        if back:
            return m.msa_qk_norm_rope_bwd_ex(None, a, None, rope, positions=pos, dx=out)[0]
        return m.msa_qk_norm_rope_ex(a, None, rope, positions=pos, out=out)

    bits = lambda t: t.view(torch.int16)    # noqa: E731
    for back in (False, True):
        clean, got = turn(x, back), turn(bad, back)
        assert torch.equal(bits(got[..., :R]), bits(clean[..., :R]))
        assert torch.equal(bits(got[..., R:]), bits(bad[..., R:])) and torch.equal(bits(clean[..., R:]), bits(x[..., R:]))
        own = bad.clone()
        assert torch.equal(bits(turn(own, back, out=own)), bits(got))
    m.msa_check_status()


@pytest.mark.parametrize("T,H,D,R,layout", ROT)
def test_norm_and_rotation_keep_channels_apart(m, T, H, D, R, layout):
    rng = np.random.default_rng(31)
    x, dy, w = (base.bf16(rng.standard_normal(s)) for s in ((T, H, D), (T, H, D), (D,)))
    rope = m.msa_rope(R, 1e6, layout=layout)
    pos = base.i32(rng.integers(0, 100000, T))
    t, h, c = T - 1, H - 1, D - 3
    bad = x.clone()
    bad[t, h, c] = math.inf
    y, clean = (m.msa_qk_norm_rope_ex(a, w, rope, positions=pos) for a in (bad, x))
    # r = 0: every other channel of the row is 0, its own is 0 * inf
    assert torch.isnan(y[t, h, c]) and (y[t, h, :c] == 0).all() and (y[t, h, c + 1:] == 0).all()
    y[t, h] = clean[t, h]
    assert torch.equal(y, clean)
    # an infinite weight of a channel that is not rotated
    wide = w.clone()
    wide[c] = math.inf
    y = m.msa_qk_norm_rope_ex(x, wide, rope, positions=pos)
    assert torch.isinf(y[..., c]).all()
    y[..., c] = clean[..., c]
    assert torch.equal(y, clean)
    # backward: dw of the other channels does not see it
    bad = dy.clone()
    bad[t, h, c] = math.inf
    (dx, dw), (cdx, cdw) = (m.msa_qk_norm_rope_bwd_ex(x, a, w, rope, positions=pos) for a in (bad, dy))
    rest = torch.arange(D, device=base.DEV) != c
    assert torch.equal(dw[rest], cdw[rest]) and not torch.isfinite(dw[c])
    dx[t, h] = cdx[t, h]
    assert torch.equal(dx, cdx)
    m.msa_check_status()
