"""The paged cache's calls where they follow, skip and refuse: calls in a row that change what the one before reads,
sequences left out, faults in the lists."""
import pytest
import torch

from paged_util import CAPACITY, LENGTH, PAGE, ROW
from test_gpu_paged import Cache, Chunk, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from medusa_tree_speculative_gb300 import build

    build.build()
    from medusa_tree_speculative_gb300 import medusa

    return medusa


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_next_call_after_a_skipped_one(M, dt):
    """Every sequence skipped (no room), in a call of two launches, then the row state changed and the call made again:
    the first one reads the old state only, so it writes nothing, time after time."""
    c = Chunk(M, dt, 4, 2, 128, 16, [20] * 60, [(b * 7) % 50 for b in range(60)], seed=41)
    before = c.k.clone(), c.v.clone()
    held = c.pages.held.clone()
    short = torch.zeros_like(held)
    length = c.pages.length.clone()
    for _ in range(50):
        c.pages.held.copy_(short)
        c.pages.length.copy_(short)
        c.run()
        c.pages.held.copy_(held)
        c.pages.length.copy_(length)
    torch.cuda.synchronize()
    assert c.err.item() == CAPACITY
    assert (c.out == 7.0).all()
    bits = torch.int16 if dt == "bf16" else torch.int32
    for p, q in zip((c.k, c.v), before):
        assert torch.equal(p.view(bits), q.view(bits))
    c.err.zero_()
    c.go()


@pytest.mark.parametrize("name,heads,order,side", [
    ("tiny_fp32", "fused", "after_lm", False), ("tiny_fp32", "split", "first", True), ("tiny_bf16", "fused", "after_lm", True),
    ("tiny_bf16", "joint", "after_accept", True), ("tiny_bf16", "fused", "after_heads", True)])
def test_sequence_without_room_is_tried_again(M, name, heads, order, side):
    """Three sequences of one closed loop (the step's own next tokens feed it), pages for the first one's tree alone: the
    others keep their trees and their output.  Once the first has ended, the same step goes on with them as a dense one
    does."""
    from medusa_tree_speculative_gb300 import step, synth, workloads
    from parity_util import to_dev

    L, ps = 21, 16
    w = dict(workloads.get(name), B=3, L=(L, L, L))
    tree = M.DeviceTree(step.build_tree(w))
    T, H, Dh = tree.T, w["H"], w["Dh"]
    x = {k: to_dev(v) for k, v in synth.make_step(w, T, 6).items()}
    wts = {k: (None if v is None else to_dev(v)) for k, v in synth.make_weights(w, 6).items()}
    given = x["tokens"].clone()
    out = [torch.full((3, 40), -5, dtype=torch.int32, device="cuda") for _ in range(2)]
    out_len = [i32([4, 0, 9]) for _ in range(2)]
    s = torch.cuda.Stream() if side else None
    dense = step.VerifyStep(w, wts, tree, max_prefix=L, heads=heads)
    dense.next_tokens.copy_(given)
    x["prefix_len"].fill_(L)
    torch.cuda.synchronize()
    dense.run(dict(x, tokens=dense.next_tokens), append=(out[0], out_len[0]))
    st = step.VerifyStep(w, wts, tree, max_prefix=L, cache="paged", heads=heads, attn_order=order)
    st.next_tokens.copy_(given)
    pages = M.Pages(4, 8, 5, ps)
    g = torch.Generator(device="cuda").manual_seed(1)
    pools = [torch.randn(5, H, ps, Dh, generator=g, device="cuda").to(x["k_cache"].dtype) for _ in range(2)]
    M.medusa_pages_reserve(pages, i32([L, L, 0, 0]), st.copies, st.n_copies, None, st.err)
    M.medusa_pages_commit(pages, None, i32([L, L, 0, 0]), 0, st.err)
    M.medusa_pages_fork(pages, i32([1]), i32([3]), st.err)
    y = dict(x, tokens=st.next_tokens, k_pages=pools[0], v_pages=pools[1], pages=pages, rows=i32([0, 3, 1]),
             n_new=i32([T, T, 0, T]))
    torch.cuda.synchronize()
    st.run(y, side_stream=s, append=(out[1], out_len[1]))
    torch.cuda.synchronize()
    A = dense.accept_len.tolist()
    assert st.err.item() == CAPACITY | ROW and st.served.tolist() == [0, -1, -1]
    assert st.accept_len.tolist() == [A[0], -1, -1]
    assert torch.equal(st.next_tokens[1:], given[1:]) and torch.equal(st.next_tokens[0], dense.next_tokens[0])
    assert out_len[1].tolist() == [4 + A[0] + 1, 0, 9] and (out[1][1:] == -5).all()
    assert torch.equal(out[1][0], out[0][0])
    # the first one ends; -1 leaves it out
    st.err.zero_()
    M.medusa_pages_free(pages, i32([0, -1, -1, -1]), st.err)
    y.update(rows=i32([-1, 3, 1]), n_new=i32([0, T, 0, T]))
    kept = st.next_tokens[0].clone()
    torch.cuda.synchronize()
    st.run(y, side_stream=s, append=(out[1], out_len[1]))
    torch.cuda.synchronize()
    assert st.err.item() == ROW and st.served.tolist() == [-1, 3, 1]
    assert st.accept_len.tolist() == [-1, A[1], A[2]]
    assert torch.equal(st.next_tokens[1:], dense.next_tokens[1:]) and torch.equal(st.next_tokens[0], kept)
    assert torch.equal(out[1], out[0]) and torch.equal(out_len[1], out_len[0])
    assert pages.length.tolist() == [0, L + A[2] + 1, 0, L + A[1] + 1]


def test_advance_by_itself(M):
    """Buffers of their own, no output, faults of the acceptance; the largest tree."""
    g = torch.Generator().manual_seed(2)
    B, T, K = 16, 512, 8
    tokens, cand = (torch.randint(0, 1000, (B, T), generator=g, dtype=torch.int32).cuda() for _ in range(2))
    nodes = torch.randint(0, T, (B, K + 1), generator=g, dtype=torch.int32)
    nodes[3, 2] = T
    alen = [b % (K + 1) for b in range(B)]
    alen[3], alen[5] = 4, K + 1
    served = [b if b % 4 else -1 for b in range(B)]
    for with_out in (True, False):
        err, out, n = i32([0]), torch.full((B, 20), -5, dtype=torch.int32, device="cuda"), i32([b for b in range(B)])
        nxt, a = torch.zeros(B, T, dtype=torch.int32, device="cuda"), i32(alen)
        M.medusa_pages_advance(i32(served), tokens, cand, nodes.cuda(), a, nxt, *((out, n) if with_out else (None, None)),
                               err)
        torch.cuda.synchronize()
        assert err.item() == (LENGTH | 2 | CAPACITY if with_out else 0)
        for b in range(B):
            on = served[b] >= 0
            assert torch.equal(nxt[b], (cand if on else tokens)[b]) and a[b] == (alen[b] if on else -1)
            if not with_out or not on or b in (3, 5) or b + alen[b] + 1 > 20:
                assert n[b] == b and (out[b] == -5).all() or b == 3
            else:
                assert n[b] == b + alen[b] + 1
                assert torch.equal(out[b, b:b + alen[b] + 1], tokens[b][nodes[b, :alen[b] + 1].long().cuda()])
    with pytest.raises(M.MedusaError, match="buffer of its own"):
        M.medusa_pages_advance(i32(served), tokens, nxt, nodes.cuda(), a, nxt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n,far", [([1, 1, 1, 1], 1), ([1] * 40, 1), ([20, 1, 30, 5], 1), ([20, 1, 30, 5], 60)])
def test_starts_that_decrease(M, dt, n, far):
    """One start behind the next one's (by one, and past every other): the call is refused whole, since its sequences'
    tokens overlap or are nobody's; with the start put back it is right."""
    c = Chunk(M, dt, 4, 2, 128, 16, n, [70] * len(n), gap=2, seed=42)
    before = c.k.clone(), c.v.clone()
    good = c.q_start.clone()
    bits = torch.int16 if dt == "bf16" else torch.int32
    for at in (1, len(n) - 1):
        c.q_start[at] = min(int(good[at + 1]) + far, c.total)
        c.run()
        torch.cuda.synchronize()
        assert c.err.item() == LENGTH
        assert (c.out == 7.0).all()
        for p, q in zip((c.k, c.v), before):
            assert torch.equal(p.view(bits), q.view(bits))
        c.q_start.copy_(good)
        c.err.zero_()
    c.go()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n", [[1, 1, 1], [20, 1, 30]])
def test_tokens_outside_the_buffers(M, dt, n):
    """Sequences that begin before the first token or end past the last one are skipped, the others are right."""
    c = Chunk(M, dt, 4, 2, 128, 16, n, [70, 5, 33], seed=43)
    before = c.k.clone(), c.v.clone()
    c.q_start[0] = -1
    c.q_start[3] = c.total + 1
    c.max_new += 1
    c.run()
    torch.cuda.synchronize()
    assert c.err.item() == LENGTH
    c.check(before, skip=(0, 2))


def test_reserve_on_a_free_tail_page(M):
    """A row whose partly filled tail page has no holder (a broken state): PAGE, not served, so that the call does not
    hand that page to another row and let both write there."""
    c = Cache(M, 3, 4, 12, 16)
    c.reserve([20, 20, 0])
    c.commit(None, [20, 20, 0])
    p = int(c.pages.table[0, 1])
    c.pages.refs[p] = 0
    c.pages.free_bits[0] |= 1 << p
    M.medusa_pages_reserve(c.pages, i32([1, 1, 40]), c.copies, c.n_copies, c.granted, c.err)
    assert c.err.item() == PAGE and c.granted.tolist() == [0, 1, 1] and c.n_copies.item() == 0
    assert c.pages.held.tolist() == [2, 2, 3] and int(c.pages.table[2, 0]) == p


def turn_fractions(pos, theta, D):
    """pos * theta^(-2j/D) / (2 pi) mod 1 for every j, from 60 decimal digits."""
    import decimal

    with decimal.localcontext() as ctx:
        ctx.prec = 60
        two_pi = 2 * decimal.Decimal("3.14159265358979323846264338327950288419716939937510582097494")
        lg = decimal.Decimal(theta).ln()
        return [float((pos * (-2 * j * lg / D).exp() / two_pi) % 1) for j in range(D // 2)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("L", [5, 2 ** 20 + 3, 2 ** 24 + 1, 2 ** 28 - 40])
def test_angles_at_far_positions(M, dt, L):
    """Up to the longest row a cache may hold (2^28 tokens, its pages all one and the same but the last): the rotation
    of the appended keys, and the result."""
    import math

    D, ps, n, theta = 64, 256, 3, 10000.0
    ty = torch.bfloat16 if dt == "bf16" else torch.float32
    most = 2 ** 28 // ps
    p = M.Pages(1, most, 2, ps)
    held = -(-(L + n) // ps)
    p.table[0, :held] = 0
    first = L // ps  # the chunk's page is the row's own
    p.table[0, first:held] = 1
    assert held - first == 1
    p.length[0], p.held[0] = L, held
    g = torch.Generator(device="cuda").manual_seed(44)
    k, v = (torch.randn(2, 1, ps, D, generator=g, device="cuda").to(ty) for _ in range(2))
    q, kn, vn = (torch.randn(n, 1, D, generator=g, device="cuda").to(ty) for _ in range(3))
    out, err = torch.zeros(n, 1, D, dtype=ty, device="cuda"), i32([0])
    ws = torch.zeros(M.medusa_paged_attn_workspace_size(1, n, n, 1, 1, D, ty), dtype=torch.uint8, device="cuda")
    M.medusa_paged_attn(q, kn, vn, k, v, p, None, i32([0, n]), n, None, theta, D ** -0.5, out, ws, err)
    torch.cuda.synchronize()
    assert err.item() == 0
    u = torch.finfo(ty).eps / 2

    def turned(x, i):
        f = torch.tensor(turn_fractions(L + i, theta, D), dtype=torch.float64, device="cuda") * (2 * math.pi)
        a, b = x[i, 0, :D // 2].double(), x[i, 0, D // 2:].double()
        return torch.cat([a * f.cos() - b * f.sin(), b * f.cos() + a * f.sin()]), (a.abs() + b.abs()).repeat(2)

    for i in range(n):
        want, size = turned(kn, i)
        got = k[1, 0, (L + i) % ps].double()
        # the angle; sine and cosine to two units in the last place, two products and a sum; the cache's rounding
        angle = 2 * math.pi * (2.0 ** -26 + (L + i) * 2.0 ** -53)
        assert ((got - want).abs() <= (angle + 2.0 ** -23 + 2 * 2.0 ** -24) * size + u * want.abs()).all(), i
        assert torch.equal(v[1, 0, (L + i) % ps], vn[i, 0])
        # a page's key counts as often as the row holds it
        kk = torch.cat([k[0, 0], k[1, 0, :(L + i) % ps + 1]]).double()
        vv = torch.cat([v[0, 0], v[1, 0, :(L + i) % ps + 1]]).double()
        times = torch.cat([torch.full((ps,), float(first), device="cuda", dtype=torch.float64),
                           torch.ones((L + i) % ps + 1, device="cuda", dtype=torch.float64)])
        z = kk @ turned(q, i)[0] * D ** -0.5 + times.log()
        w = torch.softmax(z, -1)
        # scores to 2^-18 (a bf16 query's two parts, 64 products, the angle's 2^-22); a CTA's share of tiles (of 64
        # keys, 152 CTAs at the least), added one after the other to sums and normaliser; the result's rounding
        tiles = (L + n) / 64 / 152 + 2
        tol = (2.0 ** -16 + 2 * tiles * 2.0 ** -24) * (w @ vv.abs()) + u * (w @ vv).abs()
        assert ((out[i, 0].double() - w @ vv).abs() <= tol).all(), i
