"""Attention behind a shared prefix: how exact it is beside the plain call, and what its other tests take on trust."""
import pytest
import torch

from test_gpu_paged import Chunk, M, cartesian_tree  # noqa: F401 (M is a fixture)
from test_gpu_paged_precision import bound, exact, off
from test_gpu_paged_shared import Shared, go

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


@pytest.mark.parametrize("n", [1, 30])
def test_common_tokens_come_from_one_row_whatever_the_others_name(M, n):
    """The other rows' tables name a page of NaN, which nobody holds, for the common tokens."""
    c = Shared(M, "bf16", 8, 2, 128, 16, [4], [640], [n] * 4, [5, 0, 33, 60], seed=n)
    page = c.book.refs.index(0)
    assert c.k[page].isnan().all() and c.v[page].isnan().all() and page not in sum(c.book.table, [])
    for r in c.rows[1:]:
        c.pages.table[r, :40] = page
    go(c)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("what", ["none", "single", "zero"])
def test_nothing_shared_and_the_plain_call_are_within_the_formulas_bound(M, dt, what):
    """Both, element by element."""
    sizes, P = {"none": ([], []), "single": ([1, 1], [320, 320]), "zero": ([3], [320])}[what]
    c = Shared(M, dt, 8, 2, 128, 16, sizes, P, [1, 1, 1], [5, 100, 64], 320 if what == "zero" else 0, seed=2)
    if what == "zero":
        c.common_dev.zero_()
    go(c)
    c.run = lambda: Chunk.run(c)
    go(c)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 70])
def test_calls_repeat_themselves(M, dt, n):
    """The same bits from call to call, whoever comes first."""
    c = Shared(M, dt, 8, 2, 128, 16, [16, 9], [700, 2000], [n] * 25, [37 + b for b in range(25)], seed=1)
    c.run()
    first = c.out.clone()
    for _ in range(10):
        c.out.zero_()
        c.run()
        assert torch.equal(c.out, first)
