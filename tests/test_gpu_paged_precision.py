"""How exact the chunk attention over the paged cache is: the 2-norm of its error against 64-bit formulas, relative to
the result's.  A bound on every element for itself has to allow for the worst case of thousands of roundings that in
truth average out; these ones have no such slack."""
import math

import numpy as np
import pytest
import torch

from paged_util import rotate
from test_gpu_paged import Chunk, cartesian_tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from medusa_tree_speculative_gb300 import build

    build.build()
    from medusa_tree_speculative_gb300 import medusa

    return medusa


def exact(c):
    """The batch's result in 64 bits [total][H][Dh]."""
    want = torch.zeros(c.total, c.H, c.Dh, dtype=torch.float64, device="cuda")
    for b, r in enumerate(c.rows):
        n, L, at = c.n[b], c.L[b], c.start[b]
        if n == 0:
            continue
        i = torch.arange(n, device="cuda")
        if c.tree is not None:
            pos = L + torch.from_numpy(c.tree.host.depth).cuda().long()
            words = torch.from_numpy(c.tree.host.anc_mask.view(np.int32).astype(np.int64) & 0xFFFFFFFF).cuda()
            anc = (words[:, torch.arange(n, device="cuda") // 32] >> (i % 32)) & 1
            seen = torch.cat([torch.ones(n, L, dtype=torch.bool, device="cuda"), anc.bool()], 1)
        else:
            pos = L + i
            seen = torch.arange(L + n, device="cuda")[None] <= pos[:, None]
        q = rotate(c.q[at:at + n].double(), pos, c.theta) * c.scale
        page, line = c.book.slots(r, torch.arange(L + n, device="cuda"))
        for h in range(c.H):
            hk = h // (c.H // c.Hkv)
            k, v = c.k[page, hk, line].double(), c.v[page, hk, line].double()
            z = (q[:, h] @ k.T).masked_fill(~seen, -torch.inf)
            want[at:at + n, h] = torch.softmax(z, -1) @ v
    return want


def off(c, want):
    """The kernel's relative error, and that of the exact result rounded once to the output's type."""
    c.run()
    torch.cuda.synchronize()
    assert c.err.item() == 0
    used = torch.zeros(c.total, dtype=torch.bool, device="cuda")
    for b, n in enumerate(c.n):
        used[c.start[b]:c.start[b] + n] = True
    e = [((x[used].double() - want[used]).norm() / want[used].norm()).item() for x in (c.out, want.to(c.dt))]
    return e


def bound(c, r):
    """Queries have two bf16 parts (2^-16 together) and sums 32 bits (scores up to some ten, so weights to 2^-19): the
    result is off by its own rounding, r, up to the chance of another sample (under 2% for thousands of elements), and
    by less than 2^-14 besides.  Chunks of more than 128 rows per key head round the weights once to bf16 as well: a
    rounding is uniform over a step, 2^-8 / sqrt(3) in units of the binade's lower end, and mantissas spread evenly over
    their logarithm are sqrt(3 / (2 ln 2)) such units in the mean square: 0.00153 of the weight, independent of r."""
    w = 0.00153 if max(c.n) * (c.H // c.Hkv) > 128 else 0.0
    return 1.05 * math.hypot(r, w) + 2.0 ** -14


@pytest.mark.parametrize("H,Hkv,Dh,ps,n,L", [
    (8, 2, 128, 16, [1], [1000]), (32, 8, 128, 16, [1] * 9, [3000] * 9), (32, 32, 64, 32, [1] * 3, [700, 5000, 40]),
    (16, 1, 128, 64, [1] * 5, [2000] * 5), (4, 4, 128, 16, [7, 16, 2], [100, 900, 4000]),
    (8, 4, 64, 256, [8, 3, 5], [6000, 10, 2500])])
def test_few_rows(M, H, Hkv, Dh, ps, n, L):
    c = Chunk(M, "bf16", H, Hkv, Dh, ps, n, L, seed=31)
    c.run()  # the appended keys, which `exact` reads
    e, r = off(c, exact(c))
    print(e, r)
    assert e <= bound(c, r)


CHUNKS = [  # H, Hkv, Dh, ps, n, L
    (4, 1, 128, 16, [64, 5], [0, 4000]), (8, 8, 64, 32, [70, 128], [3000, 900]), (2, 2, 128, 64, [129, 500], [2000, 40]),
    (10, 2, 64, 32, [300, 1, 41], [100, 5000, 700]), (4, 4, 128, 128, [1500], [0])]


@pytest.mark.parametrize("H,Hkv,Dh,ps,n,L", CHUNKS)
def test_chunks(M, H, Hkv, Dh, ps, n, L):
    c = Chunk(M, "bf16", H, Hkv, Dh, ps, n, L, seed=32)
    c.run()
    e, r = off(c, exact(c))
    print(e, r)
    assert e <= bound(c, r)


@pytest.mark.parametrize("s,nodes,H,Hkv,Dh", [((4, 4, 4), 64, 6, 6, 128), ((4, 4, 4), 84, 8, 4, 64),
                                             ((2, 2, 2), 14, 40, 4, 128), ((4, 4, 4, 4), 340, 2, 2, 128)])
def test_trees(M, s, nodes, H, Hkv, Dh):
    t = cartesian_tree(M, list(s), nodes)
    c = Chunk(M, "bf16", H, Hkv, Dh, 32, [t.T, t.T], [333, 4000], tree=t, seed=nodes)
    c.run()
    e, r = off(c, exact(c))
    print(e, r)
    assert e <= bound(c, r)


@pytest.mark.parametrize("H,Hkv,Dh,ps,n,L", [
    (8, 8, 64, 16, [1] * 40, [8000] * 40), (8, 8, 64, 64, [1] * 16, [30000] * 16), (16, 16, 128, 16, [1] * 20, [9000] * 20),
    (16, 4, 64, 16, [200] * 4, [6000] * 4), (8, 8, 128, 32, [150] * 4, [5000] * 4)])
def test_float32_long_prefixes(M, H, Hkv, Dh, ps, n, L):
    """Units of thousands of keys per CTA.  A score's error is that of 64 or 128 products added in turn, about 11 steps
    of 2^-25 of it, 3e-7, and every weight's as much; the sum over a tile adds 8 steps (1e-7), the sum of at most 940
    tiles 30 (weighed by their growing partial sums half of it: 4e-7), the normaliser as much.  Their squares' sum is
    the square of 6e-7, where a sum that runs over single keys would have 100 steps (3e-6)."""
    c = Chunk(M, "f32", H, Hkv, Dh, ps, n, L, seed=33)
    c.run()
    e, _ = off(c, exact(c))
    print(e)
    assert e <= 1e-6
