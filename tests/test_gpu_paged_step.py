"""The verify step and the decode loop over a paged cache, beside the same ones over dense slabs: acceptance, heads and
candidates bit for bit, the attention against 64-bit formulas, the caches line by line."""
import numpy as np
import pytest
import torch

from medusa_tree_speculative_gb300 import synth, workloads
from paged_util import attention, half_step, rotate
from parity_util import to_dev

pytestmark = pytest.mark.gpu
SAME = ("logits", "accept_len", "accepted_nodes", "next_root", "best_node", "best_logp", "head_logits", "topk",
        "next_tokens")


@pytest.fixture(scope="module")
def M():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from medusa_tree_speculative_gb300 import build

    build.build()
    from medusa_tree_speculative_gb300 import medusa

    return medusa


@pytest.mark.parametrize("name,ps,side", [("tiny_fp32", 16, False), ("tiny_bf16", 64, True),
                                          ("vicuna7b_L1024_tree64", 16, True)])
def test_step_on_pages(M, name, ps, side):
    """Row 2 of a cache continues a row that another one shares: the step copies the shared tail page first."""
    from medusa_tree_speculative_gb300 import step

    w = workloads.get(name)
    tree = M.DeviceTree(step.build_tree(w))
    T, H, Dh, L = tree.T, w["H"], w["Dh"], w["L"][0] - 3  # off a page's end
    x = {k: to_dev(v) for k, v in synth.make_step(w, T, 4).items()}
    wts = {k: (None if v is None else to_dev(v)) for k, v in synth.make_weights(w, 4).items()}
    x["prefix_len"].fill_(L)
    per = -(-(L + T) // ps)
    pages = M.Pages(3, per, 2 * per, ps)
    kp, vp = (torch.zeros(2 * per, H, ps, Dh, dtype=x["k_cache"].dtype, device="cuda") for _ in range(2))
    new = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    dense = step.VerifyStep(w, wts, tree, max_prefix=L)
    st = step.VerifyStep(w, wts, tree, max_prefix=L, cache="paged")
    M.medusa_pages_reserve(pages, new([L, 0, 0]), st.copies, st.n_copies, None, st.err)
    M.medusa_pages_commit(pages, new([0]), new([L]), 0, st.err)
    at = torch.arange(L, device="cuda")

    def lines(r, i):
        return pages.table[r, i // ps].long(), i % ps

    start = int(x["seq_start"][0])
    for pool, slab in ((kp, x["k_cache"]), (vp, x["v_cache"])):
        page, line = lines(0, at)
        pool[page, :, line] = slab[start:start + L]
    M.medusa_pages_fork(pages, new([0]), new([2]), st.err)
    before = [kp[lines(0, at)[0], :, at % ps].clone(), vp[lines(0, at)[0], :, at % ps].clone()]
    y = dict(x, k_pages=kp, v_pages=vp, pages=pages, rows=new([2]), n_new=new([0, 0, T]))
    s = [torch.cuda.Stream() for _ in range(2)] if side else [None, None]
    torch.cuda.synchronize()
    dense.run(x, side_stream=s[0])
    st.run(y, side_stream=s[1])
    torch.cuda.synchronize()
    assert st.err.item() == 0 and dense.err.item() == 0
    for f in SAME:
        assert torch.equal(getattr(st, f), getattr(dense, f)), f
    A = int(st.accept_len.item())
    assert st.n_copies.item() == 1 and pages.length.tolist() == [L, 0, L + A + 1]
    assert int(x["prefix_len"].item()) == L + A + 1
    page, line = lines(0, at)  # the row it came from is as it was
    assert torch.equal(kp[page, :, line], before[0]) and torch.equal(vp[page, :, line], before[1])
    i = torch.arange(L + A + 1, device="cuda")
    page, line = lines(2, i)
    u = half_step(kp.dtype)
    k, v = x["k_cache"][start:start + L + A + 1], x["v_cache"][start:start + L + A + 1]
    assert torch.equal(vp[page, :, line], v)
    assert torch.equal(kp[page, :, line][:L], k[:L])
    # the dense rotation's angle is a float32 product: off by up to (L + T) 2^-24 radians, each side rounds once
    off = (kp[page, :, line][L:].double() - k[L:].double()).abs()
    size = k[L:].double().abs()
    size = size + size.roll(Dh // 2, -1)
    assert (off <= 2 * u * k[L:].double().abs() + ((L + T) * 2.0 ** -23 + 2.0 ** -20) * size).all()
    # attention: the prefix and the tree's keys, before the compaction moved them
    host = tree.host
    pos = L + torch.from_numpy(host.depth).cuda().long()
    anc = torch.from_numpy(((host.anc_mask[:, np.arange(T) // 32] >> (np.arange(T) % 32).astype(np.uint32)) & 1) != 0)
    seen = torch.cat([torch.ones(T, L, dtype=torch.bool, device="cuda"), anc.cuda()], 1)
    for h in sorted({0, H // 2, H - 1}):
        q = rotate(x["q"][0, :, h:h + 1].double(), pos, 10000.0)[:, 0]
        kt = rotate(x["k_new"][0, :, h:h + 1].double(), pos, 10000.0)[:, 0].to(kp.dtype).double()
        want, tol = attention(q, torch.cat([before[0][:, h].double(), kt]),
                              torch.cat([before[1][:, h].double(), x["v_new"][0, :, h].double()]), seen, Dh ** -0.5, u,
                              L + T + Dh + 64)
        # a key's rounding to the cache's type may fall the other way
        assert ((st.out[0, :, h].double() - want).abs() <= 2 * tol).all()


@pytest.mark.parametrize("name,B,ps,graph", [("tiny_fp32", 3, 16, False), ("tiny_bf16", 2, 32, True),
                                             ("vicuna7b_L1024_tree64", 1, 256, True)])
def test_loop_on_pages(M, name, B, ps, graph):
    """Twelve chained steps emit the dense loop's tokens and keep its cache, also as replays of one captured step."""
    from medusa_tree_speculative_gb300 import loop, step

    n = 12
    w = dict(workloads.get(name), B=B)
    tree = M.DeviceTree(step.build_tree(w))
    model = loop.StandInModel(w, seed=3)
    x0 = np.array([(97 * b + 5) % w["V"] for b in range(B)])
    both = [loop.DecodeLoop(w, model, tree, n, L0=w["L"][0], x0=x0, page_size=p) for p in (None, ps)]
    side = torch.cuda.Stream()
    for _ in range(n):
        both[0].step(side_stream=side)
    paged, todo = both[1], n
    if graph:
        paged.step(side_stream=side)
        g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            paged.step(s, side_stream=side)
        todo = n - 1
    for _ in range(todo):
        g.replay() if graph else paged.step(side_stream=side)
    torch.cuda.synchronize()
    assert all(lp.st.err.item() == 0 for lp in both)
    got, want = paged.emitted(), both[0].emitted()
    pages, ps = paged.x["pages"], paged.x["pages"].page_size
    cap = int(both[0].x["seq_cap"][0])
    for b in range(B):
        assert np.array_equal(got[b], want[b])
        L = w["L"][0] + len(got[b])
        assert int(pages.length[b]) == L == int(both[0].x["prefix_len"][b])
        i = torch.arange(L, device="cuda")
        page = pages.table[b, i // ps].long()
        assert torch.equal(paged.x["v_pages"][page, :, i % ps], both[0].x["v_cache"][b * cap:b * cap + L])
    refs = pages.refs.cpu()
    assert int(refs.sum()) == int(pages.held.sum()) and refs.max() == 1


@pytest.mark.parametrize("name,ps", [("tiny_fp32", 16), ("tiny_bf16", 16)])
def test_step_without_room(M, name, ps):
    """Three sequences, pages for one tree: the first goes on, the others, which share a tail page that their trees
    would begin in, are skipped whole."""
    from medusa_tree_speculative_gb300 import step

    L = 21
    w = dict(workloads.get(name), B=3, L=(L, L, L))
    tree = M.DeviceTree(step.build_tree(w))
    T, H, Dh = tree.T, w["H"], w["Dh"]
    x = {k: to_dev(v) for k, v in synth.make_step(w, T, 5).items()}
    wts = {k: (None if v is None else to_dev(v)) for k, v in synth.make_weights(w, 5).items()}
    new = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    st = step.VerifyStep(w, wts, tree, max_prefix=L, cache="paged")
    assert 2 * ps < L + T <= 3 * ps  # each row needs one more page, the sharers a copy of their tail as well
    pages = M.Pages(4, 8, 5, ps)
    g = torch.Generator(device="cuda").manual_seed(1)
    pools = [torch.randn(5, H, ps, Dh, generator=g, device="cuda").to(x["k_cache"].dtype) for _ in range(2)]
    M.medusa_pages_reserve(pages, new([L, L, 0, 0]), st.copies, st.n_copies, None, st.err)
    M.medusa_pages_commit(pages, None, new([L, L, 0, 0]), 0, st.err)
    M.medusa_pages_fork(pages, new([1]), new([3]), st.err)
    before = pages.state.clone(), [p.clone() for p in pools]
    st.out.fill_(7.0)
    st.run(dict(x, k_pages=pools[0], v_pages=pools[1], pages=pages, rows=new([0, 3, 1]), n_new=new([T, T, 0, T])))
    torch.cuda.synchronize()
    assert st.err.item() == 4 | 64  # capacity, and rows that are skipped
    assert st.served.tolist() == [0, -1, -1]
    assert pages.length.tolist() == [L + 1 + int(st.accept_len[0]), L, 0, L]
    assert (st.out[1:] == 7.0).all() and not (st.out[0] == 7.0).any()
    others = torch.ones(5, dtype=torch.bool, device="cuda")
    others[pages.table[0, :3].long()] = False
    assert int(others.sum()) == 2
    for p, q in zip(pools, before[1]):
        assert torch.equal(p[others], q[others])
    old = M.Pages.from_state(before[0], 4, 8, 5, ps)
    assert torch.equal(pages.table[1:], old.table[1:]) and torch.equal(pages.held[1:], old.held[1:])


def kernel_nodes(run):
    """Kernels in the graph that `run(stream)` is captured into."""
    import ctypes

    g, s = torch.cuda.CUDAGraph(keep_graph=True), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        run(s)
    cu = ctypes.CDLL("libcuda.so.1")
    graph, n = ctypes.c_void_p(g.raw_cuda_graph()), ctypes.c_size_t(0)
    assert cu.cuGraphGetNodes(graph, None, ctypes.byref(n)) == 0
    nodes = (ctypes.c_void_p * n.value)()
    assert cu.cuGraphGetNodes(graph, nodes, ctypes.byref(n)) == 0
    kernels, kind = 0, ctypes.c_int(0)
    for node in nodes:
        assert cu.cuGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(kind)) == 0
        kernels += kind.value == 0
    return kernels


@pytest.mark.parametrize("name", ["tiny_fp32", "tiny_bf16"])
@pytest.mark.parametrize("s,ps", [((2, 2, 2), 16), ((3, 3, 3), 16), ((2, 2, 2), None)])
def test_launches_per_step(M, name, s, ps):
    """The kernels of a captured step of the loop, paged (trees of 15 and 40 rows, on both sides of 16) and dense."""
    from medusa_tree_speculative_gb300 import loop, step

    w = dict(workloads.get(name), tree=("cartesian", s, None))
    t = M.DeviceTree(step.build_tree(w))
    lp = loop.DecodeLoop(w, loop.StandInModel(w, seed=3), t, 4, L0=w["L"][0], x0=[5] * w["B"], page_size=ps)
    side = torch.cuda.Stream()
    lp.step(side_stream=side)
    assert kernel_nodes(lambda s: lp.step(s, side_stream=side)) == lp.launches_per_step()


@pytest.mark.parametrize("name,H,Hkv,s,side", [("tiny_bf16", 8, 2, (3, 3, 3), True), ("tiny_bf16", 2, 1, (2, 2, 2), False),
                                               ("tiny_fp32", 4, 2, (2, 2, 2), True), ("tiny_bf16", 16, 1, (1,), False)])
def test_step_with_grouped_heads(M, name, H, Hkv, s, side):
    """Query heads that share key heads (w["Hkv"]), two sequences of different lengths: the attention against 64-bit
    formulas, the accepted path's keys and values in place."""
    from medusa_tree_speculative_gb300 import step

    ps, L = 16, [21, 300]
    w = dict(workloads.get(name), B=2, H=H, Hkv=Hkv, L=L, tree=("cartesian", s, None))
    if len(s) < w["K"]:
        w["K"] = len(s)
    w["Dh"] = w["d"] // H if w["d"] // H in (64, 128) else 64
    tree = M.DeviceTree(step.build_tree(w))
    T, Dh = tree.T, w["Dh"]
    ty = step.TORCH_DT[w["dtype"]]
    x = {k: to_dev(v) for k, v in synth.make_step(w, T, 8).items()}
    wts = {k: (None if v is None else to_dev(v)) for k, v in synth.make_weights(w, 8).items()}
    g = torch.Generator(device="cuda").manual_seed(9)
    x["k_new"], x["v_new"] = (torch.randn(2, T, Hkv, Dh, generator=g, device="cuda").to(ty) for _ in range(2))
    new = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    st = step.VerifyStep(w, wts, tree, max_prefix=max(L), cache="paged")
    pages = M.Pages(3, 40, 60, ps)
    pools = [torch.full((60, Hkv, ps, Dh), float("nan"), dtype=ty, device="cuda") for _ in range(2)]
    M.medusa_pages_reserve(pages, new([L[0], 0, L[1]]), st.copies, st.n_copies, None, st.err)
    M.medusa_pages_commit(pages, None, new([L[0], 0, L[1]]), 0, st.err)
    rows = [2, 0]
    prefix = []
    for b, r in enumerate(rows):
        n = int(pages.length[r])
        i = torch.arange(n, device="cuda")
        kv = [torch.randn(n, Hkv, Dh, generator=g, device="cuda").to(ty) for _ in range(2)]
        for pool, y in zip(pools, kv):
            pool[pages.table[r, i // ps].long(), :, i % ps] = y
        prefix.append(kv)
    side_stream = torch.cuda.Stream() if side else None
    torch.cuda.synchronize()
    st.run(dict(x, k_pages=pools[0], v_pages=pools[1], pages=pages, rows=new(rows), n_new=new([T, 0, T])),
           side_stream=side_stream)
    torch.cuda.synchronize()
    assert st.err.item() == 0 and st.served.tolist() == rows
    host, u = tree.host, half_step(ty)
    anc = torch.from_numpy(((host.anc_mask[:, np.arange(T) // 32] >> (np.arange(T) % 32).astype(np.uint32)) & 1) != 0)
    for b, r in enumerate(rows):
        n = prefix[b][0].shape[0]
        pos = n + torch.from_numpy(host.depth).cuda().long()
        seen = torch.cat([torch.ones(T, n, dtype=torch.bool, device="cuda"), anc.cuda()], 1)
        q = rotate(x["q"][b].double(), pos, 10000.0)
        kt = rotate(x["k_new"][b].double(), pos, 10000.0)
        for h in range(H):
            hk = h // (H // Hkv)
            want, tol = attention(q[:, h], torch.cat([prefix[b][0][:, hk].double(), kt[:, hk].to(ty).double()]),
                                  torch.cat([prefix[b][1][:, hk], x["v_new"][b, :, hk]]).double(), seen, Dh ** -0.5, u,
                                  n + T + Dh + 64)
            # a key's rounding to the cache's type may fall the other way
            assert ((st.out[b, :, h].double() - want).abs() <= 2 * tol).all(), (b, h)
        A = int(st.accept_len[b])
        path = st.accepted_nodes[b, :A + 1].long()
        assert int(pages.length[r]) == n + A + 1
        i = torch.arange(n + A + 1, device="cuda")
        at = pages.table[r, i // ps].long(), i % ps
        k, v = pools[0][at[0], :, at[1]], pools[1][at[0], :, at[1]]
        assert torch.equal(v, torch.cat([prefix[b][1], x["v_new"][b, path]])) and torch.equal(k[:n], prefix[b][0])
        size = x["k_new"][b, path].double().abs()
        size = size + size.roll(Dh // 2, -1)
        assert ((k[n:].double() - kt[path]).abs() <= u * kt[path].abs() + 2.0 ** -21 * size).all()
