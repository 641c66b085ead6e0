"""Append, shared attention and beam selection on the GPU where values that count as equal, long
sums or overlapping storage could go wrong.  Helpers and definitions are those of
test_gpu_shared_decode.py, and so are the tolerances, in the form derived there: scores within
2^-20 + 2^-24 |score|."""
import io
import math

import numpy as np
import pytest
import torch

from oracle import shared_oracle as S
from tests import test_gpu_shared_decode as base

pytestmark = pytest.mark.gpu
m = base.m
DEV, f64, within = base.DEV, base.f64, base.within


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


# ------------------------------------------------------------------ outputs

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
