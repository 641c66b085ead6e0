"""Append, shared attention and beam selection on the GPU where values that count as equal, long
sums or overlapping storage could go wrong.  Helpers and definitions are those of
test_gpu_shared_decode.py, and so are the tolerances, in the form derived there: scores within
2^-20 + 2^-24 |score|, lse within e + 2^-22 |lse|."""
import io
import math

import numpy as np
import pytest
import torch

from oracle import shared_oracle as S
from tests import test_gpu_shared_decode as base

pytestmark = pytest.mark.gpu
m = base.m
DEV, f64, i32, bf16, within = base.DEV, base.f64, base.i32, base.bf16, base.within


# ------------------------------------------------------------------ values that count as equal

def choice(m, x, scores, W, K, **kw):
    """The very choice of the definition: for rows whose different scores are far apart."""
    so, po, to = m.msa_beam_select(x, scores, W, K, **kw)
    m.msa_check_status()
    fin = kw.get("finished")
    ws, wp, wt = S.beam_select(f64(x), f64(scores), W, K, None if fin is None else fin.cpu().numpy(), kw.get("pad_token", 0))
    assert np.array_equal(to.cpu().numpy(), wt), (to.cpu().numpy(), wt)
    assert np.array_equal(po.cpu().numpy(), wp)
    live = ws > -np.inf
    assert (f64(so)[~live] == -np.inf).all()
    within(f64(so)[live], ws[live], 2.0 ** -20 + 2.0 ** -24 * np.abs(ws[live]), "score")


def generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,K", [(4, 1), (50, 3), (5000, 16), (5000, 64), (70001, 20)])
def test_zeros_of_either_sign_are_equal(m, dt, V, K):
    g = generator(V + K)
    x = torch.full((2, V), -1.0, device=DEV)
    many = torch.rand(2, V, generator=g, device=DEV) < 0.6                  # some of these K or more
    x[many] = 0.0
    x[many & (torch.rand(2, V, generator=g, device=DEV) < 0.5)] = -0.0
    x[:, 0], x[:, 1] = -0.0, 0.0
    choice(m, x.to(dt), torch.tensor([-1.0, -1.5], device=DEV), 1, K)
    x[:, 2:] = -1.0                                                         # a few
    choice(m, x.to(dt), torch.tensor([-1.0, -1.5], device=DEV), 1, 1)


def test_scores_of_zeros_of_either_sign_are_equal(m):
    x, s = torch.zeros(6, 10, device=DEV), torch.tensor([-0.0, 0.0, -0.0, 0.0, -0.0, 0.0], device=DEV)
    fin = torch.ones(6, dtype=torch.bool, device=DEV)
    for W, K in ((2, 1), (3, 2), (6, 4), (6, 6)):
        choice(m, x, s, W, K, finished=fin, pad_token=7)


HUGE = [50, 5000, 70001, 300000]


@pytest.mark.parametrize("V", HUGE)
def test_values_above_the_limit_are_equal(m, V):
    """What lies above 2^28 counts as 2^28: the lowest places are chosen, not the largest values."""
    g = generator(V)
    x = torch.randn(3, V, generator=g, device=DEV)
    up = torch.rand(3, V, generator=g, device=DEV) < 0.5
    x = torch.where(up, 2.0 ** (29 + 90 * torch.rand(3, V, generator=g, device=DEV)), x)
    x[1, V // 2:] = math.inf
    x[2, :V // 3] = -1.0
    for dt in (torch.float32, torch.bfloat16):
        for W, K in ((1, 1), (1, 5), (3, 16)):
            choice(m, x.to(dt), torch.tensor([-1.0, -2.0, -30.0], device=DEV), W, K)
    choice(m, torch.tensor([[3e8, 4e8, 0.0, 0.0]], device=DEV), torch.zeros(1, device=DEV), 1, 1)


@pytest.mark.parametrize("V", HUGE)
def test_low_values_beside_others_keep_their_size(m, V):
    """Only where a beam has nothing else do values below -2^28 count as -2^28."""
    lows = -(2.0 ** torch.linspace(30, 120, 40, device=DEV))
    for top in (math.inf, 1e30, 2.0 ** 28, 2.0e8, 5.0, -2.0e8, -2.0 ** 28):
        x = torch.full((2, V), -math.inf, device=DEV)
        at = torch.randperm(V, generator=generator(V), device=DEV)
        x[:, at[:40]] = lows
        x[0, at[41]] = x[1, at[41]] = top
        choice(m, x, torch.tensor([-1.0, -2.0], device=DEV), 1, 9)
        choice(m, x, torch.tensor([-1.0, -2.0], device=DEV), 2, 9)


@pytest.mark.parametrize("V", HUGE)
def test_values_below_the_limit_are_equal_where_there_is_nothing_else(m, V):
    g = generator(V)
    x = -(2.0 ** (29 + 90 * torch.rand(4, V, generator=g, device=DEV)))
    x[1, torch.rand(V, generator=g, device=DEV) < 0.9] = -math.inf
    x[2] = -math.inf
    x[2, torch.randperm(V, generator=g, device=DEV)[:7]] = torch.tensor([-1e9, -3e8, -1e30, -1e9, -2e38, -2e9, -1e10], device=DEV)
    x[3, :V // 2] = math.nan
    for dt in (torch.float32, torch.bfloat16):
        for W, K in ((1, 1), (1, 20), (4, 30)):
            choice(m, x.to(dt), torch.tensor([-1.0, -2.0, -30.0, -31.0], device=DEV), W, K)
    fin = torch.tensor([False, True, False, True], device=DEV)
    choice(m, x, torch.tensor([-1.0, -2.0, -3.0, -math.inf], device=DEV), 4, 12, finished=fin, pad_token=V - 1)


@pytest.mark.parametrize("V", HUGE)
def test_rows_of_low_values_beside_other_rows(m, V):
    for top in (math.inf, 2.0e8, 5.0, -2.0 ** 28):
        x = torch.full((2, V), -math.inf, device=DEV)
        at = torch.randperm(V, generator=generator(V), device=DEV)
        x[:, at[:40]] = -(2.0 ** torch.linspace(30, 120, 40, device=DEV))
        x[0, at[41]] = top
        choice(m, x, torch.tensor([-1.0, -2.0], device=DEV), 1, 9)
        choice(m, x, torch.tensor([-1.0, -2.0], device=DEV), 2, 9)


@pytest.mark.parametrize("V", [40, 5000, 70001, 300000])
@pytest.mark.parametrize("score", [0.0, -1e9, -1e16, -1e30, -3.4028234663852886e38])
def test_logits_of_a_beam_order_it_where_its_scores_are_equal(m, V, score):
    """Scores in 64 bits of a beam far below 0, or of logits next to each other, are equal: the larger logit
    is the better one, however many slices or rows a call has."""
    g = generator(V)
    x = 1e-3 * torch.randn(2, V, generator=g, device=DEV)
    x[:, ::3] = -1.0
    x[1] *= 1e-22                                       # logits nearer to each other than the scores' steps
    s = torch.tensor([score, 2 * score if score > -1e38 else -1e38], device=DEV)
    for dt in (torch.float32, torch.bfloat16):
        y = x.to(dt)
        for W, K in ((1, 1), (1, 2), (1, 20), (2, 30)):
            if W == 2 and score == 0.0:
                continue                                # beams near each other
            po, to = S.beam_order(f64(y), f64(s), W, K)
            got = m.msa_beam_select(y, s, W, K)
            assert np.array_equal(got[2].cpu().numpy(), to) and np.array_equal(got[1].cpu().numpy(), po)
            many = m.msa_beam_select(y.repeat(100, 1), s.repeat(100), W, K)
            assert torch.equal(many[2].view(100, -1)[37], got[2].view(-1))
    m.msa_check_status()


# ------------------------------------------------------------------ sums

@pytest.mark.parametrize("dt,V,W,K", [(torch.bfloat16, 1 << 24, 64, 64), (torch.float32, 1 << 24, 3, 5), (torch.float32, (1 << 24) - 5, 16, 64),
                                      (torch.bfloat16, 3000001, 64, 64)])
def test_sums_over_the_largest_vocabularies(m, dt, V, W, K):
    """Equal logits: every partial sum is rounded in the same direction, and a row's scores are s - log V."""
    x = torch.empty(W, V, dtype=dt, device=DEV)
    x.copy_((torch.arange(W, device=DEV) * (0.69 / 64) - 0.35)[:, None])
    scores = -torch.arange(W, device=DEV) / 4.0
    so, po, to = m.msa_beam_select(x, scores, W, K)
    m.msa_check_status()
    want = -math.log(V)
    within(f64(so)[0], np.full(K, want), 2.0 ** -20 + 2.0 ** -24 * abs(want), "score")
    assert (po == 0).all() and to.tolist() == [list(range(K))]
    # each row by itself
    so, po, to = m.msa_beam_select(x, scores, 1, 1)
    m.msa_check_status()
    want = f64(scores) - math.log(V)
    within(f64(so)[:, 0], want, 2.0 ** -20 + 2.0 ** -24 * np.abs(want), "score")
    assert (to == 0).all()


@pytest.mark.parametrize("case", base.BEAMS, ids=lambda c: "-".join(map(str, c)))
def test_scores_to_half_a_step(m, case):
    N, W, V, K, dt, more, masked, ended = case
    g = generator(2 * V + K)
    x = 3 * torch.randn(N * W, V + more, generator=g, device=DEV)
    x[torch.rand(x.shape, generator=g, device=DEV) < masked] = -math.inf
    x = x.to(torch.float32 if dt == "f" else torch.bfloat16)[:, :V]
    scores = -5 * torch.rand(N * W, generator=g, device=DEV)
    fin = torch.rand(N * W, generator=g, device=DEV) < ended if ended else None
    so, po, to = m.msa_beam_select(x, scores, W, K, finished=fin, pad_token=V - 1)
    m.msa_check_status()
    every = S.beam_scores(f64(x), f64(scores), None if fin is None else fin.cpu().numpy(), V - 1)
    got, p, t = f64(so), po.cpu().numpy(), to.cpu().numpy()
    live = p >= 0
    want = every[p[live], t[live]]
    within(got[live], want, 2.0 ** -20 + 2.0 ** -24 * np.abs(want), "score")
    best = np.sort(every.reshape(N, -1), 1)[:, ::-1][:, :K]
    assert np.array_equal(live, best > -np.inf)
    within(got[live], best[live], 2.0 ** -20 + 2.0 ** -24 * np.abs(best[live]), "place")


@pytest.mark.parametrize("scale,q_gain", [(2.0 ** -64, 1.0), (2.0 ** -30, 1.0), (1.0, 1.0), (1.0, 30.0), (2.0 ** 20, 1.0), (2.0 ** 64, 1.0)])
@pytest.mark.parametrize("wide", [False, True])
def test_lse_of_small_and_large_logits(m, scale, q_gain, wide):
    table, lens, P = base.tree_table(np.random.default_rng(10), [(2, [40, 90, 128]), 300, 1, (1, [30] * 9)])
    table = base.widen(table, wide)
    rng = np.random.default_rng(11)
    q = bf16(q_gain * rng.standard_normal((len(lens), 16, 128)))
    kc, vc = (bf16(rng.standard_normal((P, 1, 128, 128))) for _ in range(2))
    o, lse = m.msa_decode_shared(q, kc, vc, i32(table), i32(lens), scale=scale)
    m.msa_check_status()
    for b, n in enumerate(lens):
        K = S.row_tokens(f64(kc), table, b, 0, n)
        z = f64(q)[b] @ K.T * scale
        want = z.max(1) + np.log(np.exp(z - z.max(1, keepdims=True)).sum(1))
        e = 2.0 ** -16 * scale * (np.abs(f64(q)[b]) @ np.abs(K).T).max() + 2.0 ** -18
        within(f64(lse)[b], want, e + 2.0 ** -22 * np.abs(want), f"lse {b}")


# ------------------------------------------------------------------ both forms of the attention

def test_shared_attention_by_items_beyond_4_gb(m):
    """Pages whose byte offsets pass 32 bits, by the kernels that read shared pages once."""
    P, Hkv = 40000, 4
    kc, vc = (torch.zeros(P, Hkv, 128, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    g = generator(8)
    pages = [39999, 33000, 12, 39000]
    for c in (kc, vc):
        c[pages] = torch.randn(4, Hkv, 128, 128, generator=g, device=DEV).to(torch.bfloat16)
    q = torch.randn(2, 16, 128, generator=g, device=DEV).to(torch.bfloat16)
    table, lens = np.array([[39999, 33000, 12], [39999, 33000, 39000]]), np.array([300, 384])
    o, lse = m.msa_decode_shared(q, kc, vc, i32(base.widen(table)), i32(lens))
    m.msa_check_status()
    t2 = np.vectorize({p: i for i, p in enumerate(pages)}.get)(table)
    want, wlse = S.attend(f64(q), f64(kc[pages]), f64(vc[pages]), t2, lens, base.SCALE)
    assert np.linalg.norm(f64(o) - want) <= 2.0 ** -8 * np.linalg.norm(want)
    within(f64(lse), wlse, 2.0 ** -10, "lse")


def test_shared_attention_by_items_equals_the_sparse_step_up_to_its_blocks(m):
    rng = np.random.default_rng(13)
    lens = [2048, 1, 700, 1999]
    table, lens, P = base.tree_table(rng, [int(n) for n in lens], maxp=16)
    q, qi = bf16(rng.standard_normal((4, 32, 128))), bf16(rng.standard_normal((4, 2, 128)))
    kc, vc, ic = (bf16(rng.standard_normal((P, 2, 128, 128))) for _ in range(3))
    a, _ = m.msa_decode_step(q, qi, kc, vc, ic, i32(table), i32(lens))
    b, _ = m.msa_decode_shared(q, kc, vc, i32(base.widen(table)), i32(lens))
    assert np.linalg.norm(f64(a) - f64(b)) <= 2.0 ** -7 * np.linalg.norm(f64(b))
    m.msa_check_status()


# ------------------------------------------------------------------ outputs

@pytest.mark.parametrize("case", [c for c in base.APPEND if c[8]], ids=lambda c: f"{len(c[0])}x{c[2]}x{c[3]}")
def test_append_in_place_with_index_heads(m, case):
    n, before, G, Hkv, R, layout, scaling, norms, _ = case
    x, w, (kc, vc, ic), table, cu, end, pos, row = base.append_case(n, before, G, Hkv, True, seed=len(n) + R)
    factor = 1.0 if scaling == "none" else 4.0
    rope = m.msa_rope(R, 1e7, layout=layout, scaling=scaling, factor=factor, orig_len=4096.0)
    wt = {k: w[k] if k in norms else None for k in "qkij"}

    def call(q, qi, caches, **out):
        return m.msa_cache_append(q, x["k"], x["v"], *caches[:2], i32(table), i32(cu), i32(end), rope, w_q=wt["q"], w_k=wt["k"],
                                  q_idx=qi, k_idx=x["k_idx"], kidx_cache=caches[2], w_qi=wt["i"], w_ki=wt["j"], **out)
    first = (kc, vc, ic)
    again = [torch.full_like(c, 7.0) for c in first]
    q, qi = call(x["q"], x["q_idx"], first)
    q2, qi2 = x["q"].clone(), x["q_idx"].clone()
    a, b = call(q2, qi2, again, q_out=q2, q_idx_out=qi2)
    m.msa_check_status()
    assert a is q2 and b is qi2 and torch.equal(q2, q) and torch.equal(qi2, qi)
    assert all(torch.equal(s, t) for s, t in zip(again, first))


def test_selected_outputs_are_tensors_of_their_own(m):
    """Saved together, grown or kept by themselves."""
    x = torch.randn(8, 1000, generator=generator(5), device=DEV)
    out = m.msa_beam_select(x, torch.zeros(8, device=DEV), 4)
    want = [t.clone() for t in out]
    buf = io.BytesIO()
    torch.save(dict(zip("spt", out)), buf)
    buf.seek(0)
    back = torch.load(buf)
    assert all(torch.equal(back[k], t) for k, t in zip("spt", want))
    assert len({t.untyped_storage().data_ptr() for t in out}) == 3
    out[0].resize_(30).fill_(5.0)
    assert torch.equal(out[1], want[1]) and torch.equal(out[2], want[2])
