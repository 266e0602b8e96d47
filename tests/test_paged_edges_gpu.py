"""Edges of the paged cache on the GPU: block scales, far positions, rotation bases, arrays out of
range, against the fp64 oracle.  Tolerances as in test_paged_gpu.py."""
import numpy as np
import pytest

import oracle
import attention_attn_fwd_08_gb300 as A
from test_paged_gpu import Cache, run_step

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,hd,page", [("e4m3", 64, 16), ("e5m2", 128, 64), ("e4m3", 256, 32), ("e5m2", 256, 16), ("e4m3", 128, 256)])
def test_single_tokens_grow_blocks_of_many_heads(kind, hd, page):
    """A token to each sequence, a warp to each block: it reads the scale that it then replaces."""
    c = Cache("bf16", kind, [9 + b % 5 for b in range(24)], 5, hd, page, seed=51)
    at = [b % 5 for b in range(24)]
    c.fill(at, 51)
    for step, spread in enumerate((1e-3, 300.0, 1e-2, 3e4, 1.0)):
        run_step(c, at, [1] * 24, spread, seed=60 + step, theta=None)
        at = [a + 1 for a in at]


@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
@pytest.mark.parametrize("new", [[1, 1, 1, 1], [9, 30, 17, 40]])
def test_append_to_blocks_of_negative_scale(kind, new):
    """A block that another program began may have a scale of either sign: one that is large enough
    stays, with the codes of the rows that are there, and one that is not grows by its magnitude."""
    before = [5, 20, 7, 3]
    c = Cache("bf16", kind, [b + n for b, n in zip(before, new)], 2, 64, 16, seed=52)
    c.fill(before, 52)
    factor = [-64.0, -1024.0, -2.0 ** -8, 1.0]
    pages = [int(c.table[b, before[b] // 16]) for b in range(4)]
    for pg, m in zip(pages, factor):
        c.ks[pg] *= m
        c.vs[pg] *= m
    old = c.host()
    run_step(c, before, new, 1.0, seed=53, theta=None)
    got = c.host()
    for b in (0, 1):  # kept: the scale, and every code under it
        n = before[b] % 16
        for w in (0, 1):
            np.testing.assert_array_equal(got[2 + w][pages[b]], old[2 + w][pages[b]])
            np.testing.assert_array_equal(got[w][pages[b], :, :n], old[w][pages[b], :, :n])
    for w in (0, 1):  # grown: a power of two, the rows' values as they were
        new_scale = got[2 + w][pages[2]]
        assert (new_scale > np.abs(old[2 + w][pages[2]])).all() and (np.log2(new_scale) % 1 == 0).all()
        v = oracle.f8_values(kind)
        before_v = v[old[w][pages[2], :, :7]] * old[2 + w][pages[2]][:, None, None]
        after_v = v[got[w][pages[2], :, :7]] * new_scale[:, None, None]
        u, tiny = {"e4m3": (2.0 ** -4, 2.0 ** -10), "e5m2": (2.0 ** -3, 2.0 ** -17)}[kind]
        assert (np.abs(after_v - before_v) <= np.maximum(u * np.abs(before_v), tiny * new_scale[:, None, None])).all()
