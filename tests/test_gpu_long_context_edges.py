"""Long-context operators on the GPU where their arithmetic or their order of steps could
go wrong: values that are not finite or far from 1, rows that grow by many pages.
Helpers, definitions and tolerances are those of test_gpu_long_context.py."""
import numpy as np
import pytest

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
