"""Long-context operators on the host: the oracle's pins, the rotation's frequencies
and the refusals of every entry point (nothing is launched)."""
import ctypes
import math

import numpy as np
import pytest
import torch

from msa_block_sparse_gb300 import api
from msa_block_sparse_gb300 import build as B
from oracle import long_oracle as L

FAKE = ctypes.c_void_p(1 << 20)     # 16-byte aligned, never dereferenced
ODD = ctypes.c_void_p((1 << 20) + 4)


@pytest.fixture(scope="module")
def lib():
    B.build()
    return api.lib()


def _err(lib):
    return lib.msa_last_error().decode()


# ------------------------------------------------------------------ oracle pins

def test_e4m3_table_is_torchs():
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    got = L.e4m3_value(np.arange(256))
    assert np.array_equal(got[~np.isnan(want)], want[~np.isnan(want)])
    assert np.array_equal(np.isnan(got), np.isnan(want))


def test_scale_rounding_is_torchs():
    x = torch.rand(20000, generator=torch.Generator().manual_seed(1), dtype=torch.float32) * 500
    x = torch.cat([x, x * 1e-3, x * 1e-5, torch.tensor(L.E4M3).float(),
                   torch.tensor((L.E4M3[1:] + L.E4M3[:-1]) / 2).float()])
    want = x.clamp(max=448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(L.nearest_even(x.double().numpy(), L.E4M3), want)


def test_code_rounding_ties_go_to_the_even_code():
    mid = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    assert L.nearest_even(np.array(mid), L.E2M1).tolist() == [0, 2, 2, 4, 4, 6, 6]
    assert L.nearest_even(np.array([0.0, 0.26, 5.01, 6.0, 7.0]), L.E2M1).tolist() == [0, 1, 7, 7, 7]


def test_held_values_are_bf16_and_requantise_to_themselves():
    rng = np.random.default_rng(0)
    x = L.bf16_round(rng.standard_normal((50, 128)) * 2.0 ** rng.integers(-8, 8, (50, 1)))
    c, s = L.quantise(x)
    v = L.held(c, s)
    assert np.array_equal(L.bf16_round(v), v)
    big = np.abs(v).reshape(50, 8, 16).max(-1) == 6 * L.e4m3_value(s)   # scale is reached
    c2, s2 = L.quantise(v)
    assert np.array_equal(s2[big], s[big])
    assert np.array_equal(L.held(c2, s2).reshape(50, 8, 16)[big], v.reshape(50, 8, 16)[big])


def test_quantisation_of_zeros_tiny_huge_and_nonfinite_blocks():
    x = np.zeros((1, 128))
    x[0, 16] = 6 * 2.0 ** -11          # / 6 = 2^-11: below half of e4m3's least 2^-9
    x[0, 32] = 1e30                    # saturates at 6 * 448
    x[0, 48] = np.inf
    x[0, 64] = np.nan
    c, s = L.quantise(x)
    v = L.held(c, s)
    assert s[0, :5].tolist() == [0, 0, 126, 127, 127]
    assert v[0, 16] == 0 and v[0, 32] == 2688 and np.isnan(v[0, 48:80]).all()


def test_rotation_layouts_agree_after_reordering():
    rng = np.random.default_rng(2)
    z, pos = rng.standard_normal((5, 3, 64)), np.array([0, 1, 7, 1000, 123456])
    f, _ = L.rope_freqs(32, 1e4)
    inter = z.copy()
    inter[..., 0:32:2], inter[..., 1:32:2] = z[..., :16], z[..., 16:32]
    a, b = L.rotate(z, pos, f, 1.3, "half"), L.rotate(inter, pos, f, 1.3, "interleaved")
    assert np.allclose(a[..., :16], b[..., 0:32:2]) and np.allclose(a[..., 16:32], b[..., 1:32:2])
    assert np.array_equal(a[..., 32:], z[..., 32:])


def test_prologue_gradients_against_differences():
    rng = np.random.default_rng(3)
    x, w, dy = rng.standard_normal((4, 2, 64)), 0.1 * rng.standard_normal(64), rng.standard_normal((4, 2, 64))
    pos = np.array([0, 3, 50, 9])
    f, g = L.rope_freqs(48, 1e4, "yarn", 4.0, 100.0)
    dx, dw = L.prologue_bwd(x, dy, w, pos, f, g, "interleaved")
    loss = lambda x, w: (L.prologue(x, w, pos, f, g, "interleaved") * dy).sum()   # noqa: E731
    h = 1e-6
    for t, hd, c in ((0, 0, 0), (1, 1, 5), (2, 0, 47), (3, 1, 60)):
        d = np.zeros_like(x)
        d[t, hd, c] = h
        assert abs((loss(x + d, w) - loss(x - d, w)) / (2 * h) - dx[t, hd, c]) < 1e-7
    for c in (0, 13, 63):
        d = np.zeros_like(w)
        d[c] = h
        assert abs((loss(x, w + d) - loss(x, w - d)) / (2 * h) - dw[c]) < 1e-7


def test_pages_oracle_keeps_counts():
    rng = np.random.default_rng(4)
    P = L.Pages(np.full((6, 4), -1), np.zeros(6, int), np.zeros(12, int), np.arange(12))
    assert P.extend([100, 0, 300, 0, 0, 0]).tolist() == [1] * 6
    assert P.table[0, 0] == 0 and P.table[2, :3].tolist() == [1, 2, 3]
    assert P.fork([0, 2, 2, 0], [1, 3, 3, 0]).tolist() == [100, 300, -1, -1]
    P.content[:] = rng.integers(0, 1000, 12)
    shared = P.content[0]
    assert P.extend([1, 1, 0, 100, 0, 0]).tolist() == [1] * 6
    # both sharers of page 0 copy it, which frees it
    assert P.ref[0] == 0 and P.content[P.table[0, 0]] == P.content[P.table[1, 0]] == shared
    assert P.free([2, 2], [129, 0]).tolist() == [171, -1]
    counts = np.zeros(12, int)
    for b in range(6):
        for j in range(P.blocks(P.lens[b])):
            counts[P.table[b, j]] += 1
    assert np.array_equal(counts, P.ref)
    _, n = P.compact()
    assert (P.ref[:n] > 0).all() and (P.ref[n:] == 0).all()


# ------------------------------------------------------------------ frequencies

@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn"])
@pytest.mark.parametrize("dim", [16, 64, 256])
def test_rope_frequencies(lib, scaling, dim):
    r = api.msa_rope(dim, 5.0e6, scaling=scaling, factor=8.0, orig_len=8192.0)
    f, gain = L.rope_freqs(dim, 5.0e6, scaling, 8.0, 8192.0)
    got = np.array(r.freqs[:dim // 2])
    assert np.allclose(got, f, rtol=1e-12, atol=0)
    assert abs(r.gain - gain) <= 2.0 ** -24 * gain
    assert all(x == 0 for x in r.freqs[dim // 2:])


def test_rope_scaling_limits(lib):
    plain = np.array(api.msa_rope(64, 1e7).freqs[:32])
    yarn = np.array(api.msa_rope(64, 1e7, scaling="yarn", factor=4.0, orig_len=32768).freqs[:32])
    # the fastest pair keeps its angle, the slowest is stretched by the factor
    assert yarn[0] == plain[0] and math.isclose(yarn[-1], plain[-1] / 4, rel_tol=1e-12)
    assert (np.diff(yarn) < 0).all()
    assert api.msa_rope(64, 1e7, scaling="yarn", factor=1.0).gain == 1.0
    assert api.msa_rope(64, 1e7, gain=0.5).gain == 0.5


@pytest.mark.parametrize("bad", [
    dict(dim=0), dict(dim=8), dict(dim=24), dict(dim=272), dict(dim=-16), dict(base=1.0),
    dict(base=float("nan")), dict(base=float("inf")), dict(layout="diagonal"),
    dict(scaling="cubic"), dict(scaling="linear", factor=0.5),
    dict(scaling="ntk", factor=float("inf")), dict(scaling="yarn", factor=2.0, orig_len=0.0),
    dict(scaling="yarn", factor=2.0, beta_fast=1.0, beta_slow=1.0), dict(gain=0.0),
    dict(gain=-1.0), dict(gain=float("nan")),
])
def test_rope_refusals(lib, bad):
    with pytest.raises((ValueError, api.MSAError)):
        api.msa_rope(**bad)


# ------------------------------------------------------------------ refusals of the C calls

def _rope(**kw):
    return ctypes.byref(api.msa_rope(**{"dim": 64, **kw}))


def test_prologue_ex_refusals(lib):
    r = _rope()

    def call(x=FAKE, y=FAKE, T=4, H=2, D=128, w=FAKE, pos=FAKE, cu=None, S=0, rope=r, eps=1e-6):
        return lib.msa_qk_norm_rope_ex(x, y, T, H, D, w, pos, cu, S, rope, eps, None)

    for code, kw in ((1, dict(x=None)), (1, dict(y=ODD)), (1, dict(w=ODD)), (1, dict(T=0)),
                     (1, dict(H=0)), (2, dict(H=257)), (2, dict(D=96)), (1, dict(pos=None)),
                     (1, dict(pos=None, cu=FAKE, S=0)), (1, dict(pos=ODD)), (1, dict(eps=-1.0)),
                     (1, dict(eps=float("nan"))), (1, dict(rope=None)),
                     (1, dict(D=64, rope=_rope(dim=128)))):
        assert call(**kw) == code, kw
        assert _err(lib)
    bent = api.msa_rope(64)
    bent.freqs[3] = float("inf")
    assert call(rope=ctypes.byref(bent)) == 1 and "frequency 3" in _err(lib)
    bent = api.msa_rope(64)
    bent.dim = 60
    assert call(rope=ctypes.byref(bent)) == 2
    bent.dim, bent.layout = 64, 2
    assert call(rope=ctypes.byref(bent)) == 1
    bent.layout, bent.gain = 0, 0.0
    assert call(rope=ctypes.byref(bent)) == 1


def test_prologue_bwd_ex_refusals(lib):
    r = _rope()
    need = lib.msa_qk_norm_rope_bwd_ex_workspace_size(4, 2, 128)
    assert need > 0 and lib.msa_qk_norm_rope_bwd_ex_workspace_size(0, 2, 128) == 0

    def call(x=FAKE, dy=FAKE, dx=FAKE, dw=FAKE, w=FAKE, ws=FAKE, n=need, D=128):
        return lib.msa_qk_norm_rope_bwd_ex(x, dy, dx, dw, 4, 2, D, w, FAKE, None, 0, r, 1e-6, ws, n, None)

    for kw in (dict(x=None), dict(dy=None), dict(dx=ODD), dict(dw=None), dict(ws=None), dict(n=need - 1)):
        assert call(**kw) == 1, kw
    assert call(D=80) == 2


def test_cache4_refusals(lib):
    def store(k=FAKE, v=FAKE, ki=FAKE, kc=FAKE, vc=FAKE, ic=FAKE, table=FAKE, cu=FAKE, start=None,
              S=1, T=4, H=2, P=8, maxp=4, g=(1.0, 1.0, 1.0)):
        return lib.msa_cache4_store(k, v, ki, kc, vc, ic, table, cu, start, S, T, H, P, maxp, *g, None)

    def load(k=FAKE, v=FAKE, ki=FAKE, kc=FAKE, vc=FAKE, ic=FAKE, table=FAKE, cu=FAKE, start=None,
             S=1, T=4, H=2, P=8, maxp=4, g=(1.0, 1.0, 1.0)):
        return lib.msa_cache4_load(kc, vc, ic, table, cu, start, S, T, H, P, maxp, *g, k, v, ki, None)

    none = dict(k=None, v=None, ki=None, kc=None, vc=None, ic=None)
    for code, kw in ((1, dict(k=None)), (1, dict(vc=None)), (1, none), (1, dict(ki=ODD)), (1, dict(ic=ODD)),
                     (1, dict(table=None)), (1, dict(cu=ODD)), (1, dict(start=ODD)), (1, dict(S=0)),
                     (1, dict(T=0)), (1, dict(H=0)), (2, dict(H=257)), (1, dict(P=0)), (1, dict(maxp=0)),
                     (2, dict(maxp=1025)), (1, dict(g=(3.0, 1.0, 1.0))), (1, dict(g=(1.0, 0.0, 1.0))),
                     (1, dict(g=(1.0, 1.0, -2.0))), (1, dict(g=(1.0, float("inf"), 1.0))),
                     (1, dict(g=(2.0 ** 65, 1.0, 1.0))), (1, dict(g=(2.0 ** -65, 1.0, 1.0)))):
        assert store(**kw) == code, kw
        assert load(**kw) == code, kw


def test_decode4_refusals(lib):
    r = _rope()
    ptrs = dict(zip(("q", "qi", "k", "v", "ki", "wq", "wqi", "wk", "wki", "kc", "vc", "ic", "table", "lens"),
                    [FAKE] * 14))

    def append(B=2, Hq=32, H=2, P=8, maxp=4, rope=r, g=(1.0, 1.0, 1.0), eps=1e-6, qo=FAKE, qio=FAKE, **kw):
        return lib.msa_decode4_append(*{**ptrs, **kw}.values(), B, Hq, H, P, maxp, rope, *g, eps, qo, qio, None)

    for name in ptrs:
        assert append(**{name: None}) == 1 and append(**{name: ODD}) == 1
    for code, kw in ((1, dict(B=0)), (1, dict(Hq=33)), (2, dict(Hq=512)), (1, dict(H=0)), (2, dict(maxp=2000)),
                     (1, dict(rope=None)), (1, dict(rope=_rope(dim=256))), (1, dict(g=(1.0, 1.0, 0.3))),
                     (1, dict(eps=-1.0)), (1, dict(qo=None)), (1, dict(qio=ODD))):
        assert append(**kw) == code, kw

    need = lib.msa_decode4_step_workspace_size(2, 32, 2, 4)
    assert need > 0 and lib.msa_decode4_step_workspace_size(2, 32, 2, 0) == 0
    sp = dict(zip(("q", "qi", "kc", "vc", "ic", "table", "lens"), [FAKE] * 7))

    def step(B=2, Hq=32, H=2, P=8, maxp=4, scale=0.1, kg=1.0, vg=1.0, n_init=0, o=FAKE, sel=None, ws=FAKE,
             n=need, **kw):
        return lib.msa_decode4_step(*{**sp, **kw}.values(), B, Hq, H, P, maxp, scale, kg, vg, n_init, o, sel,
                                    ws, n, None)

    for name in sp:
        assert step(**{name: None}) == 1 and step(**{name: ODD}) == 1
    for code, kw in ((1, dict(B=0)), (1, dict(Hq=31)), (2, dict(Hq=34)), (2, dict(maxp=1025)), (1, dict(scale=0.0)),
                     (1, dict(scale=float("nan"))), (1, dict(kg=1.5)), (1, dict(vg=0.0)), (1, dict(n_init=16)),
                     (1, dict(n_init=-1)), (1, dict(o=None)), (1, dict(sel=ODD)), (1, dict(ws=None)),
                     (1, dict(n=need - 1)), (2, dict(B=40000, n=1 << 40))):
        assert step(**kw) == code, kw


def test_pages_refusals(lib):
    one = (ctypes.c_void_p * 1)(1 << 20)
    odd = (ctypes.c_void_p * 1)((1 << 20) + 8)
    nul = (ctypes.c_void_p * 1)(0)
    size = (ctypes.c_int64 * 1)(9216)

    def fork(src=FAKE, dst=FAKE, keep=None, n=2, t=FAKE, l=FAKE, r=FAKE, B=4, P=8, m=4, out=FAKE):
        return lib.msa_pages_fork(src, dst, keep, n, t, l, r, B, P, m, out, None)

    def free(src=FAKE, keep=None, n=2, t=FAKE, l=FAKE, r=FAKE, B=4, P=8, m=4, out=FAKE):
        return lib.msa_pages_free(src, keep, n, t, l, r, B, P, m, out, None)

    for f in (fork, free):
        for code, kw in ((1, dict(src=None)), (1, dict(keep=ODD)), (1, dict(n=0)), (1, dict(t=None)),
                         (1, dict(l=ODD)), (1, dict(r=None)), (1, dict(B=0)), (1, dict(P=0)), (1, dict(m=0)),
                         (2, dict(m=1025)), (2, dict(P=(1 << 28) + 1)), (2, dict(B=(1 << 20) + 1)),
                         (1, dict(out=None))):
            assert f(**kw) == code, kw
    need = lib.msa_pages_extend_workspace_size(4, 8)

    def extend(add=FAKE, t=FAKE, l=FAKE, r=FAKE, B=4, P=8, m=4, c=one, s=size, n=1, done=FAKE, ws=FAKE, w=need):
        return lib.msa_pages_extend(add, t, l, r, B, P, m, c, s, n, done, ws, w, None)

    cneed = lib.msa_pages_compact_workspace_size(8)

    def compact(t=FAKE, l=FAKE, r=FAKE, B=4, P=8, m=4, c=one, s=size, n=1, pm=FAKE, nl=FAKE, ws=FAKE, w=cneed):
        return lib.msa_pages_compact(t, l, r, B, P, m, c, s, n, pm, nl, ws, w, None)

    for f in (extend, compact):
        for code, kw in ((1, dict(t=None)), (1, dict(B=0)), (1, dict(c=odd)), (1, dict(c=nul)), (1, dict(c=None)),
                         (1, dict(s=None)), (1, dict(s=(ctypes.c_int64 * 1)(24))),
                         (1, dict(s=(ctypes.c_int64 * 1)(0))), (1, dict(n=9)), (1, dict(n=-1)),
                         (1, dict(ws=None)), (1, dict(w=16))):
            assert f(**kw) == code, kw
    assert extend(add=None) == 1 and extend(done=ODD) == 1
    assert compact(pm=None) == 1 and compact(nl=None) == 1

    def copy(src=FAKE, dst=FAKE, n=1, P=8, c=one, s=size, nc=1):
        return lib.msa_pages_copy(src, dst, n, P, c, s, nc, None)

    for kw in (dict(src=None), dict(dst=ODD), dict(n=0), dict(P=0), dict(nc=0), dict(c=nul)):
        assert copy(**kw) == 1, kw
    assert lib.msa_pages_extend_workspace_size(0, 8) == 0
    assert lib.msa_pages_compact_workspace_size(0) == 0


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    slab = torch.zeros(2, 2, 9216, dtype=torch.uint8)
    table = torch.zeros(4, 2, dtype=torch.int32)
    rope = api.msa_rope(64)
    with pytest.raises(ValueError):
        api.msa_qk_norm_rope_ex(x, None, rope, positions=i)
    with pytest.raises(ValueError):
        api.msa_qk_norm_rope_bwd_ex(None, x, None, rope, positions=i)
    with pytest.raises(ValueError):
        api.msa_cache4_store(x, x, x, slab, slab, slab, table[:1], torch.tensor([0, 4], dtype=torch.int32))
    with pytest.raises(ValueError):
        api.msa_decode4_step(x, x, slab, slab, slab, table, i)
    with pytest.raises(ValueError):
        api.msa_pages_fork(i[:1], i[:1], table, i, torch.zeros(8, dtype=torch.int32))
    with pytest.raises(ValueError):
        api.msa_pages_copy(i, i, [slab])


def test_gains_are_three():
    with pytest.raises(ValueError, match="gains"):
        api.msa_cache4_store(None, None, None, None, None, None, None, None, gains=(1.0, 1.0))
    with pytest.raises(ValueError, match="gains"):
        api.msa_cache4_load(None, None, None, None, None, 1, gains=(1.0,))
    with pytest.raises(ValueError, match="gains"):
        api.msa_decode4_append(*[None] * 14, api.msa_rope(64), gains=(1.0, 1.0))
    with pytest.raises(ValueError, match="gains"):
        api.msa_decode4_step(*[None] * 7, gains=(1.0, 1.0, 1.0, 1.0))


def test_decode_scale_times_gain_must_be_finite(lib):
    n = lib.msa_decode4_step_workspace_size(1, 16, 1, 4)
    args = [FAKE] * 7 + [1, 16, 1, 8, 4]
    assert lib.msa_decode4_step(*args, 1e30, 2.0 ** 64, 1.0, 0, FAKE, None, FAKE, n, None) == 1
    assert b"overflows" in lib.msa_last_error()
