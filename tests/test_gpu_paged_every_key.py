"""The chunk attention over the paged cache with inputs in which every key counts (paged_count): nothing lost, doubled or
misplaced, at the lengths where a bound for Gaussian data is wider than the result."""
import numpy as np
import pytest
import torch

from paged_count import column, needles, shares, worst
from paged_util import rotate
from test_gpu_paged import SHAPES, Chunk, cartesian_tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from medusa_tree_speculative_gb300 import build

    build.build()
    from medusa_tree_speculative_gb300 import medusa

    return medusa


def positions(c, b):
    """Positions and what is seen of sequence b's tokens."""
    n, L = c.n[b], c.L[b]
    i = torch.arange(n, device="cuda")
    if c.tree is None:
        return L + i, torch.arange(L + n, device="cuda")[None] <= (L + i)[:, None]
    words = torch.from_numpy(c.tree.host.anc_mask.view(np.int32).astype(np.int64) & 0xFFFFFFFF).cuda()
    anc = (words[:, i // 32] >> (i % 32)) & 1
    return (L + torch.from_numpy(c.tree.host.depth).cuda().long(),
            torch.cat([torch.ones(n, L, dtype=torch.bool, device="cuda"), anc.bool()], 1))


def ones(x, c, heads):
    v = torch.zeros(len(x), heads, c.Dh, dtype=c.dt, device="cuda")
    v[torch.arange(len(x), device="cuda"), :, column(x, c.Dh)] = 1.0
    return v


def every_key(c, form):
    want = torch.full((c.total, c.Dh), -1.0, dtype=torch.float64, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(5)
    k0 = torch.randint(0, 2, (c.Dh,), generator=g, device="cuda").double() * 2 - 1
    if form == "even":
        c.q.zero_()
    else:
        c.kn.zero_()
    for b, r in enumerate(c.rows):
        n, L, at = c.n[b], c.L[b], c.start[b]
        if n == 0:
            continue
        pos, seen = positions(c, b)
        x = torch.arange(L, device="cuda")
        c.vn[at:at + n] = ones(L + torch.arange(n, device="cuda"), c, c.Hkv)
        used = None
        if form == "needles":
            used = torch.cat([needles(L, 100 + b), torch.zeros(n, dtype=torch.bool)]).cuda()
            # rotated, the query is 40 / sqrt(D) times k0: its score with k0 is 40
            c.q[at:at + n] = rotate((k0 * 40.0 / c.Dh ** 0.5).expand(n, c.H, c.Dh), -pos, c.theta).to(c.dt)
        if L:
            page, line = c.book.slots(r, x)
            v = ones(x, c, c.Hkv)
            if form == "needles":
                keep = used[:L, None, None]
                c.k[page, :, line] = torch.where(keep, k0.to(c.dt), 0.0).expand(L, c.Hkv, c.Dh)
                v = torch.where(keep, v, torch.randn(v.shape, generator=g, device="cuda").to(c.dt)) if used.any() else v
            c.v[page, :, line] = v
        want[at:at + n] = shares(seen, c.Dh, used)
    c.run()
    torch.cuda.synchronize()
    assert c.err.item() == 0
    for b in range(len(c.n)):
        at = slice(c.start[b], c.start[b] + c.n[b])
        for h in range(c.H):
            off = worst(c.out[at, h], want[at], c.dt) if c.n[b] else 0.0
            assert off <= 1.0, (b, h, off)


FORMS = pytest.mark.parametrize("form", ["even", "needles"])
TYPES = pytest.mark.parametrize("dt", ["bf16", "f32"])


@FORMS
@TYPES
@pytest.mark.parametrize("H,Hkv,Dh,ps", SHAPES)
def test_single_tokens(M, form, dt, H, Hkv, Dh, ps):
    every_key(Chunk(M, dt, H, Hkv, Dh, ps, [1, 0, 1, 1, 1, 1, 1, 0], [0, 9, 1, ps - 1, ps, 127, 2500, 0], gap=2), form)


@FORMS
@TYPES
@pytest.mark.parametrize("B,Hkv,L", [(1, 1, 1), (1, 2, 4000), (2, 1, 65), (9, 2, 1000), (9, 4, 900), (20, 4, 1500),
                                     (3, 8, 30000), (1, 1, 100001)])
def test_sequences_and_lengths(M, form, dt, B, Hkv, L):
    every_key(Chunk(M, dt, 4 * Hkv, Hkv, 128, 16, [1] * B, [L] + [L // 7 + b for b in range(B - 1)], seed=B), form)


@FORMS
@TYPES
@pytest.mark.parametrize("n", [3, 40])
def test_far_prefix(M, form, dt, n):
    every_key(Chunk(M, dt, 2, 1, 64, 256, [n], [100001], seed=9), form)


@FORMS
@TYPES
@pytest.mark.parametrize("H,Hkv,Dh,ps", SHAPES)
def test_chunks_and_single_tokens(M, form, dt, H, Hkv, Dh, ps):
    every_key(Chunk(M, dt, H, Hkv, Dh, ps, [1, 33, 0, 300, 2, 1, 129], [700, 0, 5, 31, 64, 4000, 130], gap=1, seed=3),
              form)


@FORMS
@TYPES
@pytest.mark.parametrize("Dh,n,L", [(128, 95, 0), (128, 96, 97), (128, 193, 5000), (64, 127, 1), (64, 1000, 24),
                                    (128, 3001, 0), (64, 600, 9000)])
def test_chunk(M, form, dt, Dh, n, L):
    every_key(Chunk(M, dt, 4, 2, Dh, 16, [n], [L], seed=n), form)


@FORMS
@TYPES
@pytest.mark.parametrize("s,nodes,H,Hkv,Dh", [((2, 2, 2), 14, 4, 4, 64), ((4, 4, 4), 84, 6, 2, 128),
                                             ((4, 4, 4, 4), 340, 2, 2, 128), ((1,), 1, 8, 1, 64),
                                             ((4, 4, 4), 64, 5, 5, 128), ((3, 3), 12, 32, 1, 128)])
def test_trees(M, form, dt, s, nodes, H, Hkv, Dh):
    t = cartesian_tree(M, list(s), nodes)
    every_key(Chunk(M, dt, H, Hkv, Dh, 32, [t.T, 0, t.T, t.T], [0, 40, 6000, 1], tree=t, seed=nodes), form)
