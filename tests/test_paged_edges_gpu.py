"""Edges of the paged cache on the GPU: block scales, far positions, rotation bases, arrays out of
range, against the fp64 oracle.  Tolerances as in test_paged_gpu.py."""
import pytest

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
