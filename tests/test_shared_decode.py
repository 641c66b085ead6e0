"""Append to 16-bit pages, attention over shared pages, beam selection and reordering of
rows on the host: the oracle's pins and the refusals of every entry point (nothing is
launched)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import msa_block_sparse_gb300 as m
from msa_block_sparse_gb300 import api
from msa_block_sparse_gb300 import build as B
from oracle import shared_oracle as S

FAKE = ctypes.c_void_p(1 << 20)     # 16-byte aligned, never dereferenced
ODD = ctypes.c_void_p((1 << 20) + 2)


@pytest.fixture(scope="module")
def lib():
    B.build()
    return api.lib()


# ------------------------------------------------------------------ oracle pins

def test_attention_oracle_is_a_library_routine():
    rng = np.random.default_rng(0)
    lens, Hkv, G = [1, 128, 300], 2, 3
    table = np.array([[4, -1, -1], [0, -1, -1], [2, 5, 1]])
    q = rng.standard_normal((3, Hkv * G, 128))
    kc, vc = rng.standard_normal((2, 6, Hkv, 128, 128))
    o, lse = S.attend(q, kc, vc, table, lens, 0.1)
    for b, L in enumerate(lens):
        pages = table[b, :S.blocks(L)]
        k, v = (torch.tensor(c[pages].transpose(1, 0, 2, 3).reshape(Hkv, -1, 128)[:, :L]).repeat_interleave(G, 0)
                for c in (kc, vc))
        qq = torch.tensor(q[b])[:, None]
        want = torch.nn.functional.scaled_dot_product_attention(qq, k, v, scale=0.1)[:, 0]
        assert np.allclose(o[b], want, rtol=1e-10, atol=1e-12)
        assert np.allclose(lse[b], torch.logsumexp((qq * k).sum(-1) * 0.1, -1), rtol=1e-12)


def test_attention_oracle_leaves_bad_pages_out():
    rng = np.random.default_rng(1)
    q = rng.standard_normal((2, 1, 128))
    kc, vc = rng.standard_normal((2, 3, 1, 128, 128))
    a = S.attend(q, kc, vc, np.array([[0, 7, 2], [-5, 3, 9]]), [300, 384], 0.1)
    b = S.attend(q, kc, vc, np.array([[0, 2, 0], [0, 0, 0]]), [128 + 44, 0], 0.1)
    assert np.allclose(a[0], b[0]) and np.allclose(a[1], b[1])


def test_beam_oracle_by_enumeration():
    rng = np.random.default_rng(2)
    x, s = rng.integers(-3, 4, (6, 5)).astype(np.float64), np.array([-1.0, -2, -1, -np.inf, 0, -1])
    fin = np.array([0, 1, 0, 0, 0, 1])
    so, po, to = S.beam_select(x, s, 3, 7, fin, pad=2)
    for n in range(2):
        every = []
        for w in range(3):
            r = 3 * n + w
            if s[r] == -np.inf:
                continue
            if fin[r]:
                every.append((-s[r], r, 2))
                continue
            p = np.exp(x[r]) / np.exp(x[r]).sum()
            every += [(-(s[r] + math.log(p[v])), r, v) for v in range(5)]
        # ties of the enumeration are exact only within a row: compare scores, then places
        every.sort()
        got = [(-a, int(b), int(c)) for a, b, c in zip(so[n], po[n], to[n]) if b >= 0]
        assert np.allclose([e[0] for e in every[:7]], [g[0] for g in got])
        assert len(got) == min(7, len(every))
    assert po[1, -1] == (-1 if 7 > 6 else po[1, -1])


def test_beam_oracle_ends():
    x = np.array([[np.finfo(np.float32).min] * 4, [-np.inf, 1.0, np.nan, -np.inf], [np.inf, 0, np.inf, 5]])
    so, po, to = S.beam_select(x, np.array([0.0, 0, 0]), 3, 8)
    # four equal ones of log(1/4), the only live token of the second row, two of log(1/2)
    assert to[0, :7].tolist() == [1, 0, 2, 0, 1, 2, 3] and po[0, :7].tolist() == [1, 2, 2, 0, 0, 0, 0]
    assert np.allclose(so[0, :7], np.log([1, 0.5, 0.5, 0.25, 0.25, 0.25, 0.25]))


def test_reorder_oracle_keeps_counts():
    rng = np.random.default_rng(3)
    lens = np.array([0, 1, 128, 129, 640])
    table, ref, at = np.full((5, 5), -1), np.zeros(20, int), 0
    for b, L in enumerate(lens):
        for j in range(S.blocks(L)):
            table[b, j], ref[at], at = at, 1, at + 1
    for _ in range(20):
        parents = rng.integers(-1, 5, 5)
        table2, lens2, ref, kept = S.reorder(parents, table, lens, ref)
        assert all(kept[b] == (0 if p < 0 else lens[p]) for b, p in enumerate(parents))
        held = [p for b in range(5) for p in table2[b, :S.blocks(lens2[b])]]
        assert np.array_equal(np.bincount(held, minlength=20) if held else np.zeros(20), ref)
        assert all((table2[b, S.blocks(lens2[b]):][:1] == -1).all() for b in range(5) if lens2[b] != lens[b])
        table, lens = table2, lens2


# ------------------------------------------------------------------ refusals

def rope():
    return m.msa_rope(64)


def test_cache_append_refusals(lib):
    good = dict(q=FAKE, k=FAKE, v=FAKE, q_idx=None, k_idx=None, w_q=None, w_k=None, w_qi=None, w_ki=None,
                k_cache=FAKE, v_cache=FAKE, kidx_cache=None, table=FAKE, cu=FAKE, lens=FAKE, S=2, T=9, Hq=4, Hkv=2,
                P=5, maxp=3, rope=ctypes.byref(rope()), eps=1e-6, q_out=FAKE, q_idx_out=None, stream=None)

    def call(**kw):
        return lib.msa_cache_append(*{**good, **kw}.values())
    bad_rope = rope()
    bad_rope.freqs[3] = math.inf
    for kw in (dict(q=None), dict(k=ODD), dict(v=None), dict(k_cache=None), dict(v_cache=ODD), dict(table=None),
               dict(cu=None), dict(lens=ODD), dict(q_out=None), dict(w_q=ODD), dict(S=0), dict(T=0), dict(T=-1),
               dict(Hq=3), dict(Hq=0), dict(Hkv=0), dict(P=0), dict(maxp=0), dict(rope=None), dict(eps=-1.0),
               dict(eps=math.nan), dict(rope=ctypes.byref(bad_rope)), dict(q_idx=FAKE), dict(k_idx=FAKE),
               dict(kidx_cache=FAKE), dict(w_qi=FAKE), dict(q_idx=FAKE, k_idx=FAKE, kidx_cache=FAKE),
               dict(q_idx=FAKE, k_idx=FAKE, kidx_cache=ODD, q_idx_out=FAKE)):
        assert call(**kw) == 1, kw
    for kw in (dict(Hq=258, Hkv=2), dict(Hkv=257, Hq=257), dict(maxp=1025), dict(Hq=256, Hkv=1, T=2 ** 31 - 1)):
        assert call(**kw) == 2, kw


def test_decode_shared_refusals(lib):
    good = dict(q=FAKE, k_cache=FAKE, v_cache=FAKE, table=FAKE, lens=FAKE, B=3, Hq=8, Hkv=2, P=5, maxp=3, scale=0.1,
                o=FAKE, lse=None, ws=FAKE, size=1 << 40, stream=None)

    def call(**kw):
        return lib.msa_decode_shared(*{**good, **kw}.values())
    for kw in (dict(q=None), dict(k_cache=ODD), dict(v_cache=None), dict(table=None), dict(lens=None), dict(o=ODD),
               dict(lse=ODD), dict(ws=None), dict(B=0), dict(Hq=7), dict(Hkv=0), dict(P=0), dict(maxp=0),
               dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf), dict(scale=2.0 ** 65),
               dict(scale=2.0 ** -65), dict(size=lib.msa_decode_shared_workspace_size(3, 8, 2, 3) - 1)):
        assert call(**kw) == 1, kw
    for kw in (dict(B=2049), dict(Hq=129, Hkv=1), dict(Hq=1026, Hkv=27), dict(maxp=1025), dict(Hkv=257, Hq=257),
               dict(P=2 ** 31 - 1)):
        assert call(**kw) == 2, kw
    assert lib.msa_decode_shared_workspace_size(2049, 8, 2, 3) == 0
    assert lib.msa_decode_shared_workspace_size(0, 8, 2, 3) == 0


def test_beam_select_refusals(lib):
    good = dict(x=FAKE, dtype=0, ld=50, scores=FAKE, fin=None, N=2, W=3, V=50, K=4, pad=0, so=FAKE, po=FAKE, to=FAKE,
                ws=FAKE, size=1 << 40, stream=None)

    def call(**kw):
        return lib.msa_beam_select(*{**good, **kw}.values())
    for kw in (dict(x=None), dict(x=ODD), dict(x=ctypes.c_void_p((1 << 20) + 1), dtype=1), dict(dtype=2), dict(dtype=-1),
               dict(ld=49), dict(scores=None), dict(scores=ODD), dict(N=0), dict(W=0), dict(V=0), dict(K=0), dict(K=-1),
               dict(pad=50), dict(pad=-1), dict(so=None), dict(po=ODD), dict(to=None), dict(ws=None),
               dict(W=1, V=3, K=4, ld=3), dict(size=lib.msa_beam_select_workspace_size(2, 3, 50, 4) - 1)):
        assert call(**kw) == 1, kw
    for kw in (dict(W=65), dict(K=65), dict(V=2 ** 24 + 1, ld=2 ** 25), dict(N=21846)):
        assert call(**kw) == 2, kw
    assert lib.msa_beam_select_workspace_size(2, 65, 50, 4) == 0


def test_pages_reorder_refusals(lib):
    good = dict(parents=FAKE, table=FAKE, lens=FAKE, ref=FAKE, B=4, P=9, maxp=5, kept=FAKE, ws=FAKE, size=1 << 30,
                stream=None)

    def call(**kw):
        return lib.msa_pages_reorder(*{**good, **kw}.values())
    for kw in (dict(parents=None), dict(table=ODD), dict(lens=None), dict(ref=None), dict(kept=ODD), dict(ws=None),
               dict(B=0), dict(P=0), dict(maxp=0), dict(size=lib.msa_pages_reorder_workspace_size(4, 5) - 1)):
        assert call(**kw) == 1, kw
    for kw in (dict(maxp=1025), dict(B=2 ** 20 + 1), dict(P=2 ** 28 + 1)):
        assert call(**{**dict(size=1 << 50), **kw}) == 2, kw


def at(k):
    return ctypes.c_void_p((1 << 20) + (k << 12))


def test_beam_select_refuses_scores_that_overlap(lib):
    """In place only where a prompt's new scores lie where its old ones were (that call is not made here:
    the workspace is refused next)."""
    def call(so, K):
        rc = lib.msa_beam_select(at(0), 0, 50, at(1), None, 2, 3, 50, K, 0, so, at(2), at(3), at(4), 0, None)
        assert rc == 1
        return lib.msa_last_error().decode()
    assert "overlaps" in call(at(1), 4) and "overlaps" in call(at(1), 2)
    assert "overlaps" in call(ctypes.c_void_p(at(1).value + 16), 3)
    assert "workspace" in call(at(1), 3) and "workspace" in call(ctypes.c_void_p(at(1).value + 32), 3)


def test_pages_reorder_refuses_arguments_that_overlap(lib):
    names = dict(parents=at(0), table=at(1), lens=at(2), ref=at(3), B=4, P=9, maxp=5, kept=at(4), ws=at(5), size=0,
                 stream=None)

    def call(**kw):
        assert lib.msa_pages_reorder(*{**names, **kw}.values()) == 1
        return lib.msa_last_error().decode()
    assert "workspace" in call()
    for kw in (dict(kept=at(0)), dict(kept=at(2)), dict(kept=ctypes.c_void_p(at(1).value + 64)), dict(kept=at(3)),
               dict(parents=at(2)), dict(parents=at(1))):
        assert "overlaps" in call(**kw), kw


def test_binding_refuses_cpu_tensors():
    t = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: m.msa_cache_append(t, t, t, t, t, i, i, i, rope()),
                 lambda: m.msa_decode_shared(t, t, t, i, i),
                 lambda: m.msa_beam_select(torch.zeros(2, 5), torch.zeros(2), 2),
                 lambda: m.msa_pages_reorder(i, i[None], i, i)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError):
        m.msa_cache_append(t, t, t, t, t, i, i, i, "rope")


def test_beam_select_refuses_outputs_that_overlap(lib):
    """parents and tokens over what other prompts' CTAs still read, outputs over each other."""
    good = dict(x=at(0), dtype=0, ld=50, scores=at(1), fin=at(2), N=2, W=3, V=50, K=3, pad=0, so=at(3), po=at(4), to=at(5),
                ws=at(6), size=0, stream=None)

    def call(**kw):
        assert lib.msa_beam_select(*{**good, **kw}.values()) == 1
        return lib.msa_last_error().decode()
    assert "workspace" in call()
    for kw in (dict(po=at(1)), dict(to=at(1)), dict(so=at(2)), dict(po=at(2)), dict(to=at(2)), dict(po=at(3)), dict(to=at(3)),
               dict(to=at(4)), dict(po=ctypes.c_void_p(at(3).value + 16)), dict(to=ctypes.c_void_p(at(4).value + 16)),
               dict(so=at(1), po=at(1)), dict(fin=ctypes.c_void_p(at(4).value + 23))):
        assert "overlap" in call(**kw), kw
    for kw in (dict(so=at(1)), dict(fin=None), dict(po=ctypes.c_void_p(at(3).value + 32)), dict(fin=ctypes.c_void_p(at(4).value + 24))):
        assert "workspace" in call(**kw), kw


def test_pages_reorder_refuses_parents_over_the_counts(lib):
    def call(ref):
        assert lib.msa_pages_reorder(at(0), at(1), at(2), ref, 4, 9, 5, at(4), at(5), 0, None) == 1
        return lib.msa_last_error().decode()
    assert "workspace" in call(at(3))
    assert "overlaps" in call(at(0))
    assert "overlaps" in call(ctypes.c_void_p(at(0).value - 32))


def test_decode_shared_workspace_follows_the_form(lib):
    """Calls that one launch serves need none; a smaller call never needs more than a larger one."""
    size = lib.msa_decode_shared_workspace_size
    assert size(4, 64, 4, 12) <= 4096 and size(1, 16, 1, 1) <= 4096
    assert size(4, 64, 4, 200) > 1 << 20 and size(64, 64, 4, 256) > 1 << 20 and size(4, 68, 4, 12) > 1 << 20
    Bs, cols = (1, 2, 3, 9, 24, 33, 50, 70, 115, 229, 300, 610, 2048), (1, 4, 8, 9, 16, 20, 21, 31, 32, 40, 41, 64, 80, 128, 129, 1024)
    for Hq, Hkv in ((16, 1), (64, 4), (8, 8)):
        got = np.array([[size(B, Hq, Hkv, c) for c in cols] for B in Bs])
        assert (got > 0).all() and (np.diff(got, axis=0) >= 0).all() and (np.diff(got, axis=1) >= 0).all()


def test_append_and_attention_refuse_outputs_that_overlap(lib):
    """q_out may be q, q_idx_out q_idx and o q; nothing else that other CTAs still read."""
    rc = rope()
    names = ("q", "k", "v", "q_idx", "k_idx")
    x = {n: at(64 * i) for i, n in enumerate(names)}              # 9 tokens of up to 4 heads: 9,216 bytes

    def append(q_out, q_idx_out):
        r = lib.msa_cache_append(x["q"], x["k"], x["v"], x["q_idx"], x["k_idx"], None, None, None, None, at(500), at(600),
                                 at(700), at(800), at(801), at(802), 2, 9, 4, 2, 5, 3, ctypes.byref(rc), 1e-6, q_out, q_idx_out, None)
        assert r == 1
        return lib.msa_last_error().decode()
    for n in ("k", "v", "q_idx", "k_idx"):
        assert "overlaps" in append(x[n], at(900)), n
    for n in ("q", "k", "v", "k_idx"):
        assert "overlaps" in append(at(900), x[n]), n
    assert "overlaps" in append(ctypes.c_void_p(x["q"].value + 256), at(900))
    assert "overlaps" in append(at(900), ctypes.c_void_p(x["q_idx"].value + 256))
    assert "overlaps" in append(at(900), at(900))

    def attend(o, lse):
        r = lib.msa_decode_shared(at(0), at(100), at(200), at(300), at(301), 3, 8, 2, 5, 3, 0.1, o, lse, at(400), 0, None)
        assert r == 1
        return lib.msa_last_error().decode()
    assert "workspace" in attend(at(0), None) and "workspace" in attend(at(10), at(20))
    assert "overlaps" in attend(ctypes.c_void_p(at(0).value + 256), None)
    assert "overlaps" in attend(at(10), at(0)) and "overlaps" in attend(at(10), at(10))
    assert "overlaps" in attend(at(10), at(301))
