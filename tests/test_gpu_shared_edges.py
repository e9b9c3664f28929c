"""Attention behind a shared prefix: how exact it is beside the plain call."""
import pytest

from test_gpu_paged import Chunk, M, cartesian_tree  # noqa: F401 (M is a fixture)
from test_gpu_paged_precision import bound, exact, off
from test_gpu_paged_shared import Shared

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,Hkv,Dh,ps,sizes,P,n", [
    (8, 2, 128, 16, [40], [1000], 1), (8, 2, 64, 32, [20, 30], [300, 4000], 1), (16, 1, 128, 16, [9, 3], [700, 2000], 1),
    (4, 4, 64, 64, [150], [500], 1), (8, 2, 128, 16, [9], [900], 20), (4, 4, 128, 16, [2, 2], [800, 3000], 128)])
def test_weights_are_as_exact_as_the_plain_calls(M, H, Hkv, Dh, ps, sizes, P, n):
    """More than 128 rows (tokens x heads) per key head in the call, at most 128 in a sequence: its weights have two bf16
    parts in the plain call, and how many other sequences there are does not change that.  (`bound` is the plain call's.)"""
    B = sum(sizes)
    c = Shared(M, "bf16", H, Hkv, Dh, ps, sizes, P, [n] * B, [7 * b % 50 for b in range(B)], seed=41)
    assert n * B * H // Hkv > 128 >= n * H // Hkv
    c.run()  # the appended keys, which `exact` reads
    want = exact(c)
    e, r = off(c, want)
    c.run = lambda: Chunk.run(c)
    print(e, r, off(c, want)[0])
    assert e <= bound(c, r)


def test_weights_of_trees_are_as_exact_as_the_plain_calls(M):
    t = cartesian_tree(M, [2, 2, 2], 14)
    c = Shared(M, "bf16", 16, 4, 128, 32, [6], [1500], [t.T] * 6, [9 * b for b in range(6)], seed=42, tree=t)
    c.run()
    e, r = off(c, exact(c))
    assert e <= bound(c, r)
