"""The paged cache's calls refuse bad arguments before any CUDA work, and the binding refuses tensors that do not fit
(no GPU needed); and the tests' own plain bookkeeping keeps its invariants."""
import ctypes as C
import random

import pytest
import torch

from paged_util import CAPACITY, ROW, Book, attention

FAKE = 0x10000  # never dereferenced: validation rejects the call first
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="host-only validation checks run without a GPU")


@pytest.fixture(scope="module")
def M():
    from medusa_tree_speculative_gb300 import build

    build.build()
    from medusa_tree_speculative_gb300 import medusa

    return medusa


def pages(M, num_pages=8, ps=16, rows=4, max_pages=2, null=None):
    p = M.medusa_pages_t(FAKE, FAKE, FAKE, FAKE, FAKE, num_pages, ps, rows, max_pages)
    if null:
        setattr(p, null, None)
    return C.byref(p)


@no_gpu
def test_pages_struct_refusals(M):
    L = M._lib
    assert L.medusa_pages_init(None, None) == -1
    for null in ("refs", "free_bits", "length", "held", "table"):
        assert L.medusa_pages_init(pages(M, null=null), None) == -1
    for ps in (0, 8, 48, 512):
        assert L.medusa_pages_init(pages(M, ps=ps), None) == -2
    for bad in ({"rows": 0}, {"rows": 1025}, {"num_pages": 0}, {"num_pages": (1 << 26) + 1}, {"max_pages": 0},
                {"max_pages": 1 << 25}):
        assert L.medusa_pages_init(pages(M, **bad), None) == -2


@no_gpu
def test_bookkeeping_refusals(M):
    L, p = M._lib, pages(M)
    assert L.medusa_pages_free(p, None, None, None) == -1
    assert L.medusa_pages_fork(p, FAKE, FAKE, -1, None, None) == -1
    assert L.medusa_pages_fork(p, FAKE, FAKE, 1025, None, None) == -1
    assert L.medusa_pages_fork(p, None, FAKE, 1, None, None) == -1
    assert L.medusa_pages_fork(p, None, None, 0, None, None) == 0
    assert L.medusa_pages_reserve(p, None, FAKE, 4, FAKE, None, None, None) == -1
    assert L.medusa_pages_reserve(p, FAKE, FAKE + 4, 4, FAKE, None, None, None) == -1
    assert L.medusa_pages_reserve(p, FAKE, FAKE, 3, FAKE, None, None, None) == -3
    assert L.medusa_pages_served(p, None, FAKE, 5, FAKE, None) == -1
    assert L.medusa_pages_served(p, FAKE, FAKE, -1, FAKE, None) == -1
    assert L.medusa_pages_served(p, FAKE, None, 2, FAKE, None) == -1
    assert L.medusa_pages_served(p, FAKE, FAKE, 2, None, None) == -1
    assert L.medusa_pages_served(p, None, None, 0, None, None) == 0
    assert L.medusa_pages_commit(p, None, FAKE, 0, 5, None, None) == -1
    assert L.medusa_pages_commit(p, FAKE, FAKE, -1, 2, None, None) == -1
    assert L.medusa_pages_commit(p, FAKE, None, 0, 2, None, None) == -1
    assert L.medusa_pages_commit(p, None, None, 0, 0, None, None) == 0
    assert L.medusa_pages_compact_workspace_size(0) == 0
    n = L.medusa_pages_compact_workspace_size(8)
    assert n >= 4 * 8
    assert L.medusa_pages_compact(p, FAKE, 4, FAKE, FAKE, n - 1, None, None) == -4
    assert L.medusa_pages_compact(p, FAKE, 4, FAKE, None, n, None, None) == -4
    assert L.medusa_pages_compact(p, None, 4, FAKE, FAKE, n, None, None) == -1
    assert L.medusa_pages_compact(p, FAKE, -1, FAKE, FAKE, n, None, None) == -1


@no_gpu
def test_pool_refusals(M):
    L = M._lib

    def copy(k=FAKE, v=FAKE, n=8, ps=16, Hkv=2, Dh=64, dt=1, copies=FAKE, nc=FAKE, most=4):
        return L.medusa_pages_copy(k, v, n, ps, Hkv, Dh, dt, copies, nc, most, None, None)

    assert copy(k=None) == -1 and copy(v=FAKE + 8) == -1 and copy(copies=None) == -1 and copy(copies=FAKE + 4) == -1
    assert copy(Dh=96) == -2 and copy(dt=2) == -2 and copy(Hkv=0) == -1 and copy(n=1 << 25, Hkv=4) == -2
    assert copy(n=0) == -1 and copy(most=-1) == -1 and copy(most=0) == 0

    def accept(p=None, B=2, Hkv=2, Dh=64, K=4, T=20, dt=1, nodes=FAKE):
        return L.medusa_paged_compact(FAKE, FAKE, p or pages(M), None, nodes, FAKE, B, Hkv, Dh, K, T, dt, None, None)

    assert accept(B=5) == -1 and accept(K=9) == -2 and accept(T=0) == -1 and accept(T=513) == -1
    assert accept(Dh=32) == -2 and accept(dt=5) == -2 and accept(nodes=None) == -1 and accept(B=0) == 0


@no_gpu
def test_attention_refusals(M):
    L = M._lib
    tree = M.medusa_tree_t(FAKE, FAKE, FAKE, FAKE, 15, 1, 3)
    for k in range(3):
        tree.s[k] = 2
    size = L.medusa_paged_attn_workspace_size(2, 10, 5, 4, 2, 64, 1)

    def attn(q=FAKE, qs=1024, ks=1024, vs=1024, kp=FAKE, p=None, rows=FAKE, qst=FAKE, B=2, total=10, new=5, t=None, H=4,
             Hkv=2, Dh=64, theta=1e4, scale=0.1, dt=1, out=FAKE, ws=FAKE, wb=size):
        return L.medusa_paged_attn(q, qs, FAKE, ks, FAKE, vs, kp, FAKE, p or pages(M), rows, qst, B, total, new, t, H, Hkv,
                                   Dh, theta, scale, dt, out, ws, wb, None, None)

    assert attn(wb=size - 1) == -4 and attn(ws=None) == -4
    assert attn(q=None) == -1 and attn(out=None) == -1 and attn(qst=None) == -1 and attn(kp=None) == -1
    assert attn(q=FAKE + 2) == -1 and attn(qs=1025) == -1 and attn(vs=1020) == -1
    assert attn(qs=128) == -1 and attn(ks=64) == -1  # tokens that overlap
    assert attn(H=5) == -2 and attn(H=130, Hkv=2) == -2 and attn(Dh=96) == -2 and attn(dt=3) == -2
    assert attn(B=1025) == -1 and attn(rows=None, B=5) == -1 and attn(total=-1) == -1 and attn(new=-1) == -1
    assert attn(theta=0.0) == -1 and attn(scale=-1.0) == -1 and attn(scale=float("nan")) == -1
    bad = M.medusa_tree_t(FAKE, FAKE, FAKE, FAKE, 15, 2, 3)
    assert attn(t=C.byref(bad)) == -1
    assert attn(B=0) == 0 and attn(total=0) == 0 and attn(new=0) == 0
    assert attn(p=pages(M, ps=24)) == -2
    assert L.medusa_paged_attn_workspace_size(-1, 10, 5, 4, 2, 64, 1) == 0


@no_gpu
def test_binding_refuses_tensors_that_do_not_fit(M):
    n = M.Pages.state_size(4, 2, 8)
    state = torch.zeros(n, dtype=torch.int32)
    p = M.Pages.from_state(state, 4, 2, 8, 16)
    assert p.table.shape == (4, 2) and p.refs.numel() == 8 and p.free_bits.numel() == 1
    for bad in (torch.zeros(n + 1, dtype=torch.int32), torch.zeros(n), torch.zeros(2 * n, dtype=torch.int32)[::2]):
        with pytest.raises(ValueError, match="state"):
            M.Pages.from_state(bad, 4, 2, 8, 16)
    with pytest.raises(ValueError, match="keep_len"):
        M.medusa_pages_free(p, torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="keep_len"):
        M.medusa_pages_free(p, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError, match="current CUDA device"):
        M.medusa_pages_free(p, torch.zeros(4, dtype=torch.int32))
    k = torch.zeros(8, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="k_pages and v_pages"):
        M.medusa_pages_copy(k, k[:4], torch.zeros(4, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
    qkv = torch.zeros(3, 8, 64, dtype=torch.bfloat16)
    args = dict(k_pages=k, v_pages=k.clone(), pages=p, rows=None, q_start=torch.zeros(3, dtype=torch.int32), max_new=2,
                tree=None, rope_theta=1e4, scale=0.1, out=torch.zeros(3, 4, 64, dtype=torch.bfloat16),
                workspace=torch.zeros(1, dtype=torch.uint8))
    with pytest.raises(ValueError, match="k_new"):
        M.medusa_paged_attn(qkv[:, :4], qkv[:, 4:7], qkv[:, 6:], **args)
    with pytest.raises(ValueError, match="q: "):
        M.medusa_paged_attn(qkv[:, :4].float(), qkv[:, 4:6], qkv[:, 6:], **args)
    with pytest.raises(ValueError, match="side by side"):
        M.medusa_paged_attn(qkv[:, ::2], qkv[:, 4:6], qkv[:, 6:], **args)
    with pytest.raises(ValueError, match="out"):
        M.medusa_paged_attn(qkv[:, :4], qkv[:, 4:6], qkv[:, 6:], **(args | {"out": torch.zeros(3, 2, 64)}))
    with pytest.raises(ValueError, match="the cache has"):
        M.medusa_paged_attn(qkv[:, :4], qkv[:, 4:6], qkv[:, 6:], **(args | {"k_pages": k[:6], "v_pages": k[:6]}))


def test_step_refuses_an_unknown_cache():
    from medusa_tree_speculative_gb300 import step, workloads

    with pytest.raises(ValueError):
        step.VerifyStep(workloads.get("tiny_fp32"), {}, None, 1, cache="slabs")


def test_book_keeps_its_invariants():
    rng = random.Random(0)
    b = Book(9, 5, 30, 16)
    for _ in range(300):
        n = [rng.choice([0, 1, 20, 50]) for _ in range(9)]
        copies, granted, err = b.reserve(n)
        assert len(granted) == 9 and not err & ROW
        b.check()
        for r in range(9):  # whoever is served writes into pages of its own
            if granted[r] and n[r]:
                assert all(b.refs[b.table[r][c]] == 1 for c in range(b.length[r] // 16, b.held[r]))
        assert not b.commit(range(9), [x if g else 0 for x, g in zip(n, granted)], 0) & ~CAPACITY
        empty = [r for r in range(9) if not b.held[r]]
        full = [r for r in range(9) if b.length[r]]
        if empty and full:
            assert b.fork([full[0]], [empty[0]]) == 0
        b.free([rng.choice([-1, -1, -1, 0, 17]) for _ in range(9)])
        b.compact()
        b.check()
        live = sum(x > 0 for x in b.refs)
        assert all(b.refs[:live]) and not any(b.refs[live:])


def test_plain_attention_of_a_row_without_keys():
    g = torch.Generator().manual_seed(0)
    q, k, v = (torch.randn(n, 8, generator=g, dtype=torch.float64) for n in (2, 3, 3))
    out, tol = attention(q, k, v, torch.tensor([[True, True, False], [False, False, False]]), 1.0, 2.0 ** -8, 20)
    assert (out[1] == 0).all() and torch.isfinite(tol).all()
    p = torch.softmax(q[0] @ k[:2].T, -1)
    assert torch.allclose(out[0], p @ v[:2])


def test_device_errors_have_names(M):
    """The binding names every bit of the header, each fault its own."""
    import re
    from pathlib import Path

    text = (Path(__file__).resolve().parent.parent / "include" / "medusa.h").read_text()
    bits = {int(v): n for n, v in re.findall(r"MEDUSA_DEVERR_(\w+) = (\d+)", text)}
    assert bits == M.DEVERR
    assert [n for v, n in sorted(bits.items())] == ["TOKEN", "NODE", "CAPACITY", "LENGTH", "TIMEOUT", "PAGE", "ROW",
                                                    "LAYOUT"]
    assert sorted(bits) == [1 << k for k in range(len(bits))]


@no_gpu
def test_advance_refusals(M):
    L = M._lib
    bufs = [FAKE + 4096 * k for k in range(8)]

    def adv(null=None, B=2, T=20, K=4, cap=30, cand=bufs[2], out=bufs[6], out_len=bufs[7]):
        p = [bufs[0], bufs[1], cand, bufs[3], bufs[4], bufs[5]]
        if null is not None:
            p[null] = None
        return L.medusa_pages_advance(*p[:5], B, T, K, p[5], out, out_len, cap, None, None)

    assert [adv(null=k) for k in range(6)] == [-1] * 6
    assert adv(out_len=None) == -1 and adv(cap=0) == -1 and adv(cand=bufs[1]) == -1 and adv(cand=bufs[5]) == -1
    assert adv(B=0) == -1 and adv(B=17) == -1 and adv(T=0) == -1 and adv(T=513) == -1 and adv(K=9) == -1 and adv(K=-1) == -1
