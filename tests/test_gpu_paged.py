"""The paged cache on the GPU: its bookkeeping against a row-by-row implementation on lists (bit for bit), and the chunk
attention against 64-bit formulas within the bound that its roundings allow."""
import random

import numpy as np
import pytest
import torch

from paged_util import CAPACITY, LENGTH, NODE, PAGE, ROW, Book, attention, half_step, rotate

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def M():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from medusa_tree_speculative_gb300 import build

    build.build()
    from medusa_tree_speculative_gb300 import medusa

    return medusa


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Cache:
    """A cache on the GPU and its Book, changed together."""

    def __init__(self, M, rows, max_pages, num_pages, ps):
        self.M, self.book = M, Book(rows, max_pages, num_pages, ps)
        self.pages = M.Pages(rows, max_pages, num_pages, ps)
        self.err = i32([0])
        self.copies, self.n_copies, self.granted = i32([[-9] * 4] * rows), i32([-1]), i32([-1] * rows)

    def same(self, err=0):
        assert int(self.err.item()) == err
        self.err.zero_()
        got, want = self.pages.state.cpu(), self.book.state()
        assert torch.equal(got, want), (got != want).nonzero().flatten().tolist()[:20]

    def free(self, keep):
        e = self.book.free(keep)
        self.M.medusa_pages_free(self.pages, i32(keep), self.err)
        self.same(e)

    def fork(self, src, dst):
        e = self.book.fork(src, dst)
        self.M.medusa_pages_fork(self.pages, i32(src), i32(dst), self.err)
        self.same(e)

    def reserve(self, n_new, pools=()):
        copies, granted, e = self.book.reserve(n_new)
        self.M.medusa_pages_reserve(self.pages, i32(n_new), self.copies, self.n_copies, self.granted, self.err)
        self.same(e)
        assert self.n_copies.item() == len(copies) and self.granted.tolist() == granted
        assert self.copies[:len(copies)].tolist() == copies
        for k, v in pools:
            self.M.medusa_pages_copy(k, v, self.copies, self.n_copies, self.err)
        return copies, granted

    def commit(self, rows, n_new, bias=0):
        e = self.book.commit(range(len(n_new)) if rows is None else rows, n_new, bias)
        self.M.medusa_pages_commit(self.pages, None if rows is None else i32(rows), i32(n_new), bias, self.err)
        self.same(e)


# ------------------------------------------------------------ bookkeeping ---

@pytest.mark.parametrize("rows,max_pages,num_pages,ps", [(1, 1, 1, 16), (5, 3, 9, 16), (40, 20, 333, 32),
                                                         (1024, 9, 4000, 16), (64, 40, 40000, 256)])
def test_bookkeeping_random_rounds(M, rows, max_pages, num_pages, ps):
    rng = random.Random(rows)
    c = Cache(M, rows, max_pages, num_pages, ps)
    c.same()
    top = max_pages * ps
    for step in range(8):
        n_new = [rng.choice([0, 1, rng.randint(0, ps), rng.randint(0, top // 2 + 1), rng.randint(-1, top + 1)])
                 for _ in range(rows)]
        _, granted = c.reserve(n_new)
        c.commit(None, [n if g and n > 0 else 0 for n, g in zip(n_new, granted)])
        empty = [r for r in range(rows) if c.book.length[r] == 0 and c.book.held[r] == 0]
        full = [r for r in range(rows) if c.book.length[r]]
        rng.shuffle(empty)
        if empty and full:
            pairs = [(rng.choice(full), d) for d in empty[:rng.randint(1, len(empty))]]
            c.fork([s for s, _ in pairs], [d for _, d in pairs])
        if rows <= 64:
            c.book.check()
        c.free([rng.choice([-1, -1, 0, rng.randint(0, top)]) for _ in range(rows)])
        moves = c.book.compact()
        copies, n = i32([[-7] * 4] * (len(moves) + 2)), i32([-1])
        ws = torch.empty(M.medusa_pages_compact_workspace_size(num_pages), dtype=torch.uint8, device="cuda")
        M.medusa_pages_compact(c.pages, copies, n, ws, c.err)
        c.same()
        assert n.item() == len(moves) and copies[:len(moves)].tolist() == moves
        assert (copies[len(moves):] == -7).all()


def test_bookkeeping_of_a_large_pool(M):
    """Several words of the bit map per thread, the last ones ragged; a compaction that moves thousands of pages."""
    rng = random.Random(9)
    rows, most, num, ps = 30, 9000, 200013, 16
    c = Cache(M, rows, most, num, ps)
    n_new = [rng.randint(0, most * ps) for _ in range(rows)]
    c.reserve(n_new)
    c.commit(None, n_new)
    c.free([rng.choice([-1, -1, 0, rng.randint(0, n)]) for n in n_new])
    moves = c.book.compact()
    copies, n = i32([[-7] * 4] * (len(moves) + 1)), i32([-1])
    ws = torch.empty(M.medusa_pages_compact_workspace_size(num), dtype=torch.uint8, device="cuda")
    M.medusa_pages_compact(c.pages, copies, n, ws, c.err)
    c.same()
    assert len(moves) > 1000 and n.item() == len(moves) and copies.tolist() == moves + [[-7] * 4]
    c.reserve([rng.randint(0, 40) for _ in range(rows)])


def test_compact_with_a_table_that_names_free_pages(M):
    """A row whose table names a free page past the live ones: PAGE, that entry stays, the others move."""
    c = Cache(M, 3, 4, 64, 16)
    c.reserve([64, 64, 64])
    c.commit(None, [64, 64, 64])
    c.free([0, -1, -1])
    c.pages.table[1, 2] = 60
    copies, n = i32([[-7] * 4] * 8), i32([-1])
    ws = torch.empty(M.medusa_pages_compact_workspace_size(64), dtype=torch.uint8, device="cuda")
    M.medusa_pages_compact(c.pages, copies, n, ws, c.err)
    assert c.err.item() == PAGE and n.item() == 4
    assert c.pages.table[1].tolist() == [4, 5, 60, 7] and c.pages.table[2].tolist() == [0, 1, 2, 3]


def test_optional_outputs_may_be_left_out(M):
    c = Cache(M, 2, 2, 3, 16)
    M.medusa_pages_reserve(c.pages, i32([20, 40]), c.copies, c.n_copies)  # the second row does not fit
    M.medusa_pages_commit(c.pages, None, i32([20, 1]))
    M.medusa_pages_fork(c.pages, i32([0]), i32([5]))
    M.medusa_pages_free(c.pages, i32([17, -1]))
    assert c.pages.length.tolist() == [17, 0] and c.pages.held.tolist() == [2, 0]


def test_every_row_shares_one_tail(M):
    """1024 rows on one partly filled page: all but the last sharer copy it, in row order."""
    c = Cache(M, 1024, 2, 1100, 16)
    c.reserve([5] + [0] * 1023)
    c.commit([0], [5])
    c.fork([0] * 1023, list(range(1023, 0, -1)))
    copies, _ = c.reserve([1] * 1024)
    assert len(copies) == 1023 and copies[-1][3] == 1022


def test_reserve_when_pages_run_out(M):
    c = Cache(M, 6, 4, 7, 16)
    _, granted = c.reserve([16, 40, 0, 64, 1, 0])
    assert granted == [1, 1, 1, 0, 0, 0]
    c.reserve([0, 0, 0, 33, 0, 0])
    c.reserve([0, 0, 0, 0, 1, 0])


def test_fork_refusals(M):
    c = Cache(M, 8, 4, 30, 16)
    c.reserve([20, 7, 0, 0, 0, 0, 0, 0])
    c.commit(None, [20, 7, 0, 0, 0, 0, 0, 0])
    c.fork([0, 0, 1, 0, 5, 9, 0], [2, 2, 0, 1, 4, 3, -1])  # twice, taken, chained, out of range
    c.fork([0, 2, 3], [6, 7, 5])
    c.fork([6, 7], [7, 3])


def test_commit_refusals(M):
    c = Cache(M, 4, 2, 8, 16)
    c.reserve([10, 10, 10, 10])
    c.commit([3, 1, 3, 0, 4, -1], [4, 16, 5, 17, 1, 1])
    c.commit([0, 1], [-1, 0], 1)


def test_compact_list_too_short(M):
    c = Cache(M, 3, 4, 64, 16)
    c.reserve([64, 64, 64])
    c.free([0, -1, -1])
    before = c.pages.state.clone()
    copies, n = i32([[-7] * 4] * 3), i32([-1])
    ws = torch.empty(M.medusa_pages_compact_workspace_size(64), dtype=torch.uint8, device="cuda")
    M.medusa_pages_compact(c.pages, copies, n, ws, c.err)
    assert n.item() == 0 and c.err.item() == CAPACITY and torch.equal(before, c.pages.state)


def test_broken_rows_are_reported(M):
    """Pages outside the pool and impossible lengths raise PAGE; the other rows are served."""
    c = Cache(M, 4, 3, 12, 16)
    c.reserve([20, 20, 20, 20])
    c.commit(None, [20, 20, 20, 20])
    c.pages.table[1, 1] = 12
    c.pages.table[2, 0] = -5
    c.pages.length[3] = 99
    M.medusa_pages_reserve(c.pages, i32([20, 1, 0, 1]), c.copies, c.n_copies, c.granted, c.err)
    assert c.err.item() == PAGE and c.granted.tolist() == [1, 0, 1, 0]
    c.err.zero_()
    M.medusa_pages_free(c.pages, i32([-1, 0, 0, 0]), c.err)
    assert c.err.item() == PAGE and c.pages.held.tolist() == [3, 0, 0, 2]
    assert c.pages.refs.min().item() >= 0


@pytest.mark.parametrize("dt,Hkv,Dh,ps", [("bf16", 3, 64, 16), ("f32", 2, 128, 64), ("bf16", 8, 128, 256)])
def test_pages_copy(M, dt, Hkv, Dh, ps):
    g = torch.Generator(device="cuda").manual_seed(ps)
    n = 40
    pools = [torch.randn(n, Hkv, ps, Dh, generator=g, device="cuda", dtype=DT[dt]) for _ in range(2)]
    want = [p.clone() for p in pools]
    rng = random.Random(1)
    ids = rng.sample(range(n), 20)
    lines = [[ids[2 * i], ids[2 * i + 1], rng.choice([0, 1, ps // 2 + 1, ps]), 0] for i in range(10)]
    for p in want:
        for a, z, m, _ in lines:
            p[z, :, :m] = p[a, :, :m]
    bad = [[n, 0, 1, 0], [0, -1, 1, 0], [0, 1, ps + 1, 0], [1, 0, -1, 0]]
    err = i32([0])
    M.medusa_pages_copy(*pools, i32(lines + [[0, 1, ps, 0]]), i32([10]), err)
    assert err.item() == 0 and all(torch.equal(a, b) for a, b in zip(pools, want))
    M.medusa_pages_copy(*pools, i32(bad), i32([4]), err)
    assert err.item() == PAGE and all(torch.equal(a, b) for a, b in zip(pools, want))
    err.zero_()
    M.medusa_pages_copy(*pools, i32([[0, 0, 0, 0]]), i32([5]), err)
    assert err.item() == CAPACITY and all(torch.equal(a, b) for a, b in zip(pools, want))


# --------------------------------------------------------------- attention ---

def cartesian_tree(M, s, max_nodes):
    paths, plen = M.medusa_tree_cartesian(s, max_nodes)
    return M.DeviceTree(M.medusa_tree_compile(paths, plen, len(s)))


class Chunk:
    """A batch over a cache with prefixes L and new tokens n, everything around it poisoned with NaN."""

    def __init__(self, M, dt, H, Hkv, Dh, ps, n, L, tree=None, seed=0, gap=0, spread=1.0, shuffle=True, spare=4,
                 far=None):
        self.M, self.H, self.Hkv, self.Dh, self.ps, self.n, self.L = M, H, Hkv, Dh, ps, n, L
        self.tree, self.dt, self.theta, self.scale = tree, DT[dt], 10000.0, Dh ** -0.5
        rng = random.Random(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        B = len(n)
        rows = B + 2 if shuffle else B
        self.rows = rng.sample(range(rows), B) if shuffle else list(range(B))
        most = max(1, max(-(-(a + b) // ps) for a, b in zip(n, L)))
        num = far or sum(-(-(a + b) // ps) for a, b in zip(n, L)) + spare
        self.book = Book(rows, most, num, ps)
        order = rng.sample(range(num), num) if far is None else list(range(num - 1, -1, -1))
        for b, r in enumerate(self.rows):
            self.book.length[r], self.book.held[r] = L[b], -(-(L[b] + n[b]) // ps)
            for c in range(self.book.held[r]):
                self.book.table[r][c] = order.pop(0)
                self.book.refs[self.book.table[r][c]] = 1
        self.pages = M.Pages.from_state(self.book.state().cuda(), rows, most, num, ps)
        nan = float("nan")
        self.k = torch.full((num, Hkv, ps, Dh), nan, dtype=self.dt, device="cuda")
        self.v = torch.full_like(self.k, nan)
        for b, r in enumerate(self.rows):
            if L[b]:
                page, line = self.book.slots(r, torch.arange(L[b], device="cuda"))
                self.k[page, :, line] = (torch.randn(L[b], Hkv, Dh, generator=g, device="cuda") * spread).to(self.dt)
                self.v[page, :, line] = torch.randn(L[b], Hkv, Dh, generator=g, device="cuda").to(self.dt)
        # `gap` tokens before and after the sequences belong to none of them
        self.total = sum(n) + 2 * gap
        qkv = torch.randn(self.total, H + 2 * Hkv + 1, Dh, generator=g, device="cuda").to(self.dt)
        qkv[:gap] = nan
        qkv[self.total - gap:] = nan
        self.q, self.kn, self.vn = qkv[:, 1:H + 1], qkv[:, H + 1:H + 1 + Hkv], qkv[:, H + 1 + Hkv:]
        self.start = [gap + sum(n[:b]) for b in range(B + 1)]
        self.out = torch.full((self.total, H, Dh), 7.0, dtype=self.dt, device="cuda")
        self.err = i32([0])
        self.max_new = max(n)
        self.ws = torch.zeros(M.medusa_paged_attn_workspace_size(B, self.total, self.max_new, H, Hkv, Dh, self.dt),
                              dtype=torch.uint8, device="cuda")
        self.q_start, self.where = i32(self.start), i32(self.rows)

    def run(self, stream=None):
        self.M.medusa_paged_attn(self.q, self.kn, self.vn, self.k, self.v, self.pages, self.where, self.q_start,
                                 self.max_new, self.tree, self.theta, self.scale, self.out, self.ws, self.err, stream)

    def check(self, before=None, skip=()):
        """Outputs, appended keys and values, and everything that has to be as it was."""
        k0, v0 = before
        u = half_step(self.dt)
        k1, v1 = self.k.clone(), self.v.clone()
        for b, r in enumerate(self.rows):
            n, L, at = self.n[b], self.L[b], self.start[b]
            if n == 0 or b in skip:
                continue
            i = torch.arange(n, device="cuda")
            if self.tree is not None:
                pos = L + torch.from_numpy(self.tree.host.depth).cuda().long()
                words = torch.from_numpy(self.tree.host.anc_mask.view(np.int32).astype(np.int64) & 0xFFFFFFFF).cuda()
                anc = (words[:, torch.arange(n, device="cuda") // 32] >> (i % 32)) & 1
                seen = torch.cat([torch.ones(n, L, dtype=torch.bool, device="cuda"), anc.bool()], 1)
            else:
                pos = L + i
                seen = torch.arange(L + n, device="cuda")[None] <= (L + i)[:, None]
            page, line = self.book.slots(r, L + i)
            kr = rotate(self.kn[at:at + n].double(), pos, self.theta)
            # two products of 32 bits and an angle within 2^-23, then the rounding to the cache's type
            size = self.kn[at:at + n].double().abs()
            size = size + size.roll(self.Dh // 2, -1)
            assert ((self.k[page, :, line].double() - kr).abs() <= u * kr.abs() + 2.0 ** -21 * size).all()
            assert torch.equal(self.v[page, :, line], self.vn[at:at + n])
            k1[page, :, line] = k0[page, :, line]
            v1[page, :, line] = v0[page, :, line]
            q = rotate(self.q[at:at + n].double(), pos, self.theta)
            page, line = self.book.slots(r, torch.arange(L + n, device="cuda"))
            for h in range(self.H):
                hk = h // (self.H // self.Hkv)
                kh, vh = self.k[page, hk, line].double(), self.v[page, hk, line].double()
                want, tol = attention(q[:, h], kh, vh, seen, self.scale, u, L + n + self.Dh + 64)
                off = ((self.out[at:at + n, h].double() - want).abs() / tol).max().item()
                assert off <= 1.0, (b, h, off)
        # NaN compares by bits
        bits = torch.int16 if self.dt == torch.bfloat16 else torch.int32
        assert torch.equal(k1.view(bits), k0.view(bits)) and torch.equal(v1.view(bits), v0.view(bits))
        outside = torch.ones(self.total, dtype=torch.bool, device="cuda")
        for b in range(len(self.n)):
            if b not in skip:
                outside[self.start[b]:self.start[b] + self.n[b]] = False
        assert (self.out[outside] == 7.0).all()

    def go(self):
        before = self.k.clone(), self.v.clone()
        self.run()
        torch.cuda.synchronize()
        assert self.err.item() == 0
        self.check(before)


SHAPES = [  # H, Hkv, Dh, ps
    (4, 4, 128, 16), (8, 2, 128, 64), (5, 1, 64, 32), (14, 2, 128, 256), (16, 1, 64, 16), (64, 1, 128, 128),
    (6, 2, 64, 128),
]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("H,Hkv,Dh,ps", SHAPES)
def test_decode(M, dt, H, Hkv, Dh, ps):
    """One token per sequence, from an empty prefix to thousands of keys, beside sequences without tokens."""
    Chunk(M, dt, H, Hkv, Dh, ps, [1, 0, 1, 1, 1, 1, 1, 0], [0, 9, 1, ps - 1, ps, 127, 2500, 0], gap=2).go()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("H,Hkv,Dh,ps", SHAPES)
def test_mixed_batch(M, dt, H, Hkv, Dh, ps):
    """Chunks and single tokens in one batch."""
    Chunk(M, dt, H, Hkv, Dh, ps, [1, 33, 0, 300, 2, 1, 129], [700, 0, 5, 31, 64, 1, 130], gap=1, seed=3).go()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n,L", [(1, 0), (2, 0), (17, 0), (127, 1), (128, 0), (129, 128), (257, 1000), (1000, 24)])
def test_one_chunk(M, dt, n, L):
    Chunk(M, dt, 4, 2, 128, 16, [n], [L], seed=n).go()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("s,nodes,H,Hkv,Dh", [((2, 2, 2), 14, 4, 4, 64), ((4, 4, 4), 84, 6, 2, 128),
                                             ((4, 4, 4, 4), 340, 2, 2, 128), ((1,), 1, 8, 1, 64),
                                             ((3, 3), 12, 32, 1, 128)])
def test_tree(M, dt, s, nodes, H, Hkv, Dh):
    t = cartesian_tree(M, list(s), nodes)
    Chunk(M, dt, H, Hkv, Dh, 32, [t.T, 0, t.T, t.T], [0, 40, 333, 1], tree=t, seed=nodes).go()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_peaked_scores(M, dt):
    """Scores of several hundred: the running maximum moves often and weights underflow."""
    Chunk(M, dt, 4, 2, 128, 16, [1, 150], [900, 700], seed=5, spread=40.0).go()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_many_sequences(M, dt):
    n = [1] * 200 + [3] * 56
    Chunk(M, dt, 4, 4, 64, 16, n, [(b * 37) % 191 for b in range(256)], seed=6).go()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_largest_batch(M, dt):
    Chunk(M, dt, 1, 1, 64, 16, [1] * 1024, [b % 40 for b in range(1024)], seed=7, shuffle=False).go()


def test_offsets_past_32_bits(M):
    """Pages in the last megabytes of pools of 5 GB: byte offsets past 2^32."""
    c = Chunk(M, "bf16", 8, 8, 128, 16, [1, 70], [100, 60], seed=8, far=160000)
    assert c.k.numel() * 2 > 2 ** 32
    c.go()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_long_positions(M, dt):
    """Far positions: the angle stays exact (one sequence, two heads, a hundred thousand keys)."""
    Chunk(M, dt, 2, 1, 64, 256, [3], [100001], seed=9).go()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n", [[1, 1, 1], [40, 1, 200]])
def test_same_bits_every_time(M, dt, n):
    """Joins of shared units do not depend on which CTA comes last; the counters are ready again; a captured call
    replays; another shape may use the workspace in between."""
    c = Chunk(M, dt, 8, 2, 128, 16, n, [3000, 17, 900], seed=10)
    c.go()
    want = c.out.clone()
    other = Chunk(M, dt, 4, 4, 64, 32, [1, 20], [700, 300], seed=11)
    if other.ws.numel() < c.ws.numel():
        other.ws = c.ws
    for _ in range(5):
        c.out.fill_(0)
        c.run()
        assert torch.equal(c.out, want)
    other.go()
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        c.run()
    for _ in range(3):
        c.out.fill_(0)
        g.replay()
        assert torch.equal(c.out, want)
    # two calls at once, each with its own workspace, on their own streams
    d = Chunk(M, dt, 8, 2, 128, 16, n, [3000, 17, 900], seed=10)
    torch.cuda.synchronize()
    s2 = torch.cuda.Stream()
    for _ in range(4):
        c.run(s)
        d.run(s2)
    torch.cuda.synchronize()
    assert torch.equal(c.out, want) and torch.equal(d.out, want) and c.err.item() == 0 and d.err.item() == 0


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_skipped_sequences(M, dt):
    """A row named twice or out of range, pages that do not reach, a chunk longer than max_new: reported, skipped, and
    the others are right."""
    c = Chunk(M, dt, 4, 2, 128, 16, [3, 1, 20, 1, 30], [10, 50, 7, 33, 12], seed=12)
    before = c.k.clone(), c.v.clone()
    c.rows[3] = c.rows[1]
    c.where = i32(c.rows)
    c.run()
    torch.cuda.synchronize()
    assert c.err.item() == ROW
    c.check(before, skip=(3,))
    for rows3 in (-1, 7, 1 << 30):
        c = Chunk(M, dt, 4, 2, 128, 16, [3, 1, 20, 1, 30], [10, 50, 7, 33, 12], seed=12)
        before = c.k.clone(), c.v.clone()
        c.rows[3] = rows3
        c.where = i32(c.rows)
        c.run()
        assert c.err.item() == ROW
        c.check(before, skip=(3,))
    c = Chunk(M, dt, 4, 2, 128, 16, [3, 1, 20, 1, 30], [10, 50, 7, 33, 12], seed=12)
    before = c.k.clone(), c.v.clone()
    c.max_new = 20
    c.pages.held[c.rows[0]] -= 1  # 10 tokens in no page: a broken state
    c.pages.length[c.rows[1]] = -1
    c.pages.held[c.rows[2]] -= 1  # 7 tokens in one page, no room for 20 more
    c.run()
    assert c.err.item() == LENGTH | PAGE | CAPACITY
    c.check(before, skip=(0, 1, 2, 4))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n", [[1, 1], [40, 30]])
def test_page_outside_the_pool(M, dt, n):
    """A bad page of the prefix and one of the chunk: PAGE, nothing written there, zeros read; the other sequence is
    untouched by it."""
    c = Chunk(M, dt, 4, 2, 128, 16, n, [100, 60], seed=13)
    before = c.k.clone(), c.v.clone()
    c.pages.table[c.rows[0], 2] = c.pages.num_pages
    c.pages.table[c.rows[0], 6] = -3
    c.run()
    torch.cuda.synchronize()
    assert c.err.item() == PAGE
    c.out[:n[0]] = 7.0
    keep = c.book.slots(c.rows[0], torch.arange(100, 100 + n[0], device="cuda"))
    c.k[keep[0], :, keep[1]], c.v[keep[0], :, keep[1]] = before[0][keep[0], :, keep[1]], before[1][keep[0], :, keep[1]]
    c.check(before, skip=(0,))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("H,Hkv,Dh", [(2, 2, 128), (4, 1, 64), (2, 1, 128)])
@pytest.mark.parametrize("rows", [15, 16, 17, 127, 128, 129, 192])
def test_rows_around_a_tile(M, dt, H, Hkv, Dh, rows):
    """Query rows per key head (tokens x shared heads) on both sides of a tile of 16 and of 128."""
    n = max(1, rows // (H // Hkv))
    Chunk(M, dt, H, Hkv, Dh, 32, [n, 1, n], [200, 0, 1500], gap=1, seed=rows).go()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("B,Hkv,L", [(1, 1, 0), (1, 1, 1), (1, 2, 4000), (2, 1, 65), (9, 2, 1000), (9, 4, 900),
                                     (20, 4, 1500), (3, 8, 30000)])
def test_decode_sequences_and_lengths(M, dt, B, Hkv, L):
    """One token: few sequences, whose keys several CTAs share, to many; one much longer than the rest."""
    Chunk(M, dt, 4 * Hkv, Hkv, 128, 16, [1] * B, [L] + [L // 7 + b for b in range(B - 1)], seed=B).go()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_skipped_single_tokens(M, dt):
    """As test_skipped_sequences, one token each."""
    c = Chunk(M, dt, 4, 2, 128, 16, [1, 1, 1, 1, 0], [900, 50, 7, 33, 12], seed=15)
    before = c.k.clone(), c.v.clone()
    c.rows[3] = c.rows[1]
    c.where = i32(c.rows)
    c.pages.length[c.rows[2]] = -1
    c.run()
    torch.cuda.synchronize()
    assert c.err.item() == ROW | PAGE
    c.check(before, skip=(2, 3))
    c = Chunk(M, dt, 4, 2, 128, 16, [1, 1, 1, 3, 0], [900, 50, 15, 33, 12], seed=16)
    before = c.k.clone(), c.v.clone()
    c.max_new = 2
    c.pages.length[c.rows[2]] = 16  # no page for the next token
    c.run()
    torch.cuda.synchronize()
    assert c.err.item() == LENGTH | CAPACITY
    c.check(before, skip=(2, 3))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_nothing_to_do(M, dt):
    """No sequences, no tokens, only sequences without tokens: nothing is written."""
    c = Chunk(M, dt, 4, 2, 128, 16, [0, 0], [40, 0], gap=3, seed=17)
    before = c.k.clone(), c.v.clone()
    for max_new in (0, 1, 7, 300):
        c.max_new = max_new
        c.run()
    c.q_start, c.where = i32([0]), i32([])
    c.run()
    torch.cuda.synchronize()
    assert c.err.item() == 0
    c.check(before)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_long_batch_of_chunks(M, dt):
    """Thousands of new tokens in one call, one of its rows named twice."""
    c = Chunk(M, dt, 2, 1, 64, 64, [3000, 1, 2500, 700], [10, 77, 0, 129], gap=1, seed=18)
    before = c.k.clone(), c.v.clone()
    c.rows[3] = c.rows[0]
    c.where = i32(c.rows)
    c.run()
    torch.cuda.synchronize()
    assert c.err.item() == ROW
    c.check(before, skip=(3,))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 20, 150])
def test_non_finite_inputs_stay_where_they_are(M, dt, n):
    """NaN and infinities in one token's query, in a key that earlier tokens do not see, and in another sequence's
    values: every other output keeps its bits."""
    c = Chunk(M, dt, 4, 2, 128, 16, [n, n, n], [300, 40, 700], seed=19)
    c.run()
    want, err = c.out.clone(), c.err.item()
    assert err == 0
    at = c.start[0] + n // 2
    c.q[at] = float("nan")
    c.kn[c.start[2] - 1] = float("inf")
    c.vn[c.start[2] + n // 3] = float("-inf")
    c.run()
    torch.cuda.synchronize()
    same = torch.ones(3 * n, dtype=torch.bool, device="cuda")
    same[at] = same[c.start[2] - 1] = False
    same[c.start[2]:] = False
    assert torch.equal(c.out[same], want[same])
    assert c.out[at].isnan().all() and not c.out[c.start[2] + n - 1].isfinite().any()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 70])
def test_rows_left_out(M, dt, n):
    """rows = None is row b for sequence b, in a cache with more rows."""
    c = Chunk(M, dt, 4, 2, 64, 16, [n, n, 1], [33, 500, 20], seed=20, shuffle=False)
    c.go()
    want = c.out.clone()
    big = M.Pages(9, c.pages.max_pages, c.pages.num_pages, 16)
    for f in ("refs", "free_bits"):
        getattr(big, f).copy_(getattr(c.pages, f))
    for f in ("length", "held", "table"):
        getattr(big, f)[:3] = getattr(c.pages, f)
    c.pages, c.where = big, None
    c.out.fill_(7.0)
    c.run()
    torch.cuda.synchronize()
    assert c.err.item() == 0 and torch.equal(c.out, want)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 5])
def test_many_heads(M, dt, n):
    Chunk(M, dt, 300, 300, 64, 16, [n, 0, n], [70, 9, 3], seed=21).go()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_room_for_much_more(M, dt):
    """Rows whose tables reach far past what they hold."""
    for n, L in (([1, 1], [100, 3]), ([30, 1], [100, 3])):
        c = Chunk(M, dt, 8, 2, 128, 16, n, L, seed=22)
        before = c.k.clone(), c.v.clone()
        p = M.Pages(c.pages.rows, 70000, c.pages.num_pages, 16)
        for f in ("refs", "free_bits", "length", "held"):
            getattr(p, f).copy_(getattr(c.pages, f))
        p.table[:, :c.pages.max_pages] = c.pages.table
        c.pages = p
        c.run()
        torch.cuda.synchronize()
        assert c.err.item() == 0
        c.check(before)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_graphs_that_share_a_workspace(M, dt):
    """Two captured calls of different kinds with one workspace, replayed in turn on one stream."""
    a = Chunk(M, dt, 8, 2, 128, 16, [1, 1, 1], [3000, 17, 900], seed=23)
    b = Chunk(M, dt, 8, 2, 128, 16, [200, 1, 90], [300, 17, 900], seed=24)
    a.ws = b.ws
    want, graphs = [], []
    for c in (a, b):
        c.go()
        want.append(c.out.clone())
        g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            c.run()
        graphs.append(g)
    for _ in range(4):
        for c, g, w in zip((a, b), graphs, want):
            c.out.fill_(7.0)
            g.replay()
            assert torch.equal(c.out, w)
    assert a.err.item() == 0 and b.err.item() == 0


# ------------------------------------------------------------ accepted path ---

@pytest.mark.parametrize("dt,Hkv,Dh,ps", [("bf16", 4, 128, 16), ("f32", 2, 64, 32), ("bf16", 7, 64, 256)])
def test_paged_compact(M, dt, Hkv, Dh, ps):
    rng = random.Random(ps)
    T, K, B = 40, 8, 9
    L = [rng.randint(0, 100) for _ in range(B)]
    c = Chunk(M, dt, Hkv, Hkv, Dh, ps, [T] * B, L, seed=14)
    g = torch.Generator(device="cuda").manual_seed(1)
    c.k, c.v = (torch.randn(c.k.shape, generator=g, device="cuda").to(c.dt) for _ in range(2))
    alen = [0, 8, 3, 9, 2, 1, 4, -1, 2]
    nodes = [[0] + sorted(rng.sample(range(1, T), K)) for _ in range(B)]
    nodes[2] = [0, 1, 2, 3] + [-1] * 5
    nodes[4] = [0, 1, T] + [-1] * 6
    nodes[5] = [0, 0] + [-1] * 7
    rows = list(c.rows)
    rows[8] = rows[6]
    want = [c.k.clone(), c.v.clone()]
    for b in (0, 1, 2, 6):
        for p in want:
            page, line = c.book.slots(rows[b], L[b] + torch.tensor(nodes[b][:alen[b] + 1], device="cuda"))
            to, at = c.book.slots(rows[b], L[b] + torch.arange(alen[b] + 1, device="cuda"))
            p[to, :, at] = p[page, :, line].clone()
    M.medusa_paged_compact(c.k, c.v, c.pages, i32(rows), i32(nodes), i32(alen), T, c.err)
    torch.cuda.synchronize()
    assert c.err.item() == LENGTH | NODE | ROW
    assert torch.equal(c.k, want[0]) and torch.equal(c.v, want[1])
    assert torch.equal(c.pages.state.cpu(), c.book.state())


# ------------------------------------------------------------ all together ---

@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_serving_run(M, dt):
    """Prompts in chunks, forks, single tokens, a verified tree, rows that end, a compacted pool: after every step the
    cache equals a plain one that keeps each row's keys and values in a list, and the attention is right."""
    H, Hkv, Dh, ps, rows = 4, 2, 64, 16, 6
    u = half_step(DT[dt])
    c = Cache(M, rows, 20, 80, ps)
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = (torch.full((80, Hkv, ps, Dh), float("nan"), dtype=DT[dt], device="cuda") for _ in range(2))
    plain = [[torch.zeros(0, Hkv, Dh, device="cuda", dtype=DT[dt]) for _ in range(2)] for _ in range(rows)]
    ws = torch.zeros(M.medusa_paged_attn_workspace_size(rows, 400, 100, H, Hkv, Dh, DT[dt]), dtype=torch.uint8,
                     device="cuda")

    def held_equal():
        for r in range(rows):
            page, line = c.book.slots(r, torch.arange(c.book.length[r], device="cuda"))
            assert torch.equal(k[page, :, line], plain[r][0]) and torch.equal(v[page, :, line], plain[r][1])

    def chunk(where, n, tree=None, accept=None):
        n_new = [0] * rows
        for r, m in zip(where, n):
            n_new[r] = m
        _, granted = c.reserve(n_new, [(k, v)])
        assert all(granted)
        total = sum(n)
        q, kn, vn = (torch.randn(total, h, Dh, generator=g, device="cuda").to(DT[dt]) for h in (H, Hkv, Hkv))
        out = torch.zeros(total, H, Dh, dtype=DT[dt], device="cuda")
        start = [sum(n[:b]) for b in range(len(n) + 1)]
        M.medusa_paged_attn(q, kn, vn, k, v, c.pages, i32(where), i32(start), max(n), tree, 10000.0, Dh ** -0.5, out,
                            ws, c.err)
        for b, r in enumerate(where):
            L, i = c.book.length[r], torch.arange(n[b], device="cuda")
            pos = L + (torch.from_numpy(tree.host.depth).cuda().long() if tree else i)
            page, line = c.book.slots(r, L + i)
            kr = rotate(kn[start[b]:start[b + 1]].double(), pos, 10000.0)
            vr = torch.cat([plain[r][1], vn[start[b]:start[b + 1]]])
            assert ((k[page, :, line].double() - kr).abs() <= u * kr.abs() + 2.0 ** -18).all()
            assert torch.equal(v[page, :, line], vr[L:])
            page, line = c.book.slots(r, torch.arange(L + n[b], device="cuda"))
            kc = k[page, :, line]
            if tree:
                anc = torch.tensor([[(int(tree.host.anc_mask[x, y // 32]) >> (y % 32)) & 1 for y in range(tree.T)]
                                    for x in range(tree.T)], dtype=torch.bool, device="cuda")
                seen = torch.cat([torch.ones(n[b], L, dtype=torch.bool, device="cuda"), anc], 1)
            else:
                seen = torch.arange(L + n[b], device="cuda")[None] <= (L + i)[:, None]
            qr = rotate(q[start[b]:start[b + 1]].double(), pos, 10000.0)
            for h in range(H):
                want, tol = attention(qr[:, h], kc[:, h // 2].double(), vr[:, h // 2].double(), seen, Dh ** -0.5, u,
                                      L + n[b] + Dh + 64)
                assert ((out[start[b]:start[b + 1], h].double() - want).abs() <= tol).all()
            if tree:
                path = L + torch.tensor(accept[b], device="cuda")
                plain[r] = [torch.cat([plain[r][0], kc[path]]), torch.cat([plain[r][1], vr[path]])]
            else:
                plain[r] = [kc, vr]
        if tree:
            K = max(len(x) for x in accept) - 1
            nodes, alen = i32([x + [-1] * (K + 1 - len(x)) for x in accept]), [len(x) - 1 for x in accept]
            M.medusa_paged_compact(k, v, c.pages, i32(where), nodes, i32(alen), tree.T, c.err)
            c.commit(where, alen, 1)
        else:
            c.commit(where, n)
        held_equal()

    chunk([4, 1], [100, 37])
    chunk([4], [50])
    chunk([1, 4], [1, 1])
    c.fork([4, 1, 4], [0, 3, 5])
    plain[0], plain[3], plain[5] = plain[4], plain[1], plain[4]
    held_equal()
    t = cartesian_tree(M, [3, 2, 2], 21)
    paths = []
    for leaf in (t.T - 1, 0, 4, 2, 9):
        p = [leaf]
        while p[0]:
            p.insert(0, int(t.host.parent[p[0]]))
        paths.append(p)
    chunk([0, 1, 3, 4, 5], [t.T] * 5, t, paths)
    c.free([-1, 0, -1, 20, -1, 60])
    plain[1] = [x[:0] for x in plain[1]]
    plain[3], plain[5] = [x[:20] for x in plain[3]], [x[:60] for x in plain[5]]
    held_equal()
    moves = c.book.compact()
    copies, n = i32([[0] * 4] * 80), i32([0])
    w2 = torch.empty(M.medusa_pages_compact_workspace_size(80), dtype=torch.uint8, device="cuda")
    M.medusa_pages_compact(c.pages, copies, n, w2, c.err)
    M.medusa_pages_copy(k, v, copies, n, c.err)
    c.same()
    assert len(moves) > 0
    held_equal()
    chunk([0, 3, 5, 4], [1, 1, 1, 1])
    chunk([2, 3], [60, 5])
