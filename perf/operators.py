"""The paged cache's operators: what is measured, and their plain forms.

A paged cache is a pool of pages k_pages, v_pages [num_pages][Hkv][page_size][Dh] and five int32 arrays, kept side by
side in one buffer ("meta"): refs [num_pages], free_bits [ceil(num_pages / 32)], length [rows], held [rows] and table
[rows][max_pages].  Token x of row r lies in page table[r][x / page_size], line x % page_size.

Operators ("op" of a case):
  attn    medusa_paged_attn: a chunk of new tokens per sequence is rotated, appended to its pages, and attends to the
          row's cache and, causally or along a candidate tree, to itself.
  pages   medusa_pages_free, fork, reserve, copy, commit: one scheduling round of a server that frees finished rows,
          forks running ones and makes room for their next tokens, shared tail pages being copied first.
  compact medusa_pages_compact and medusa_pages_copy: the live pages move to the front of the pool.
  accept  medusa_paged_compact and medusa_pages_commit: the accepted path of a verified tree moves into place.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
THETA = 10000.0


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # One new token of one sequence at the 7B shape (32 heads of 128, prefix 1024): the smallest decode step.
        {"name": "decode_one_1024", "op": "attn", "dtype": "bf16", "H": 32, "Hkv": 32, "Dh": 128, "ps": 16, "B": 1,
         "n_lo": 1, "n_hi": 1, "L_lo": 1024, "L_hi": 1024, "T": 0, "lens": 1},
        # One new token for each of 64 ragged sequences, four query heads to a key head: a decode batch of a server.
        {"name": "decode_batch64", "op": "attn", "dtype": "bf16", "H": 32, "Hkv": 8, "Dh": 128, "ps": 16, "B": 64,
         "n_lo": 1, "n_hi": 1, "L_lo": 500, "L_hi": 8192, "T": 0, "lens": 2},
        # A prompt of 8192 tokens in one chunk: prefill, the largest amount of arithmetic.
        {"name": "prefill_8192", "op": "attn", "dtype": "bf16", "H": 32, "Hkv": 8, "Dh": 128, "ps": 64, "B": 1,
         "n_lo": 8192, "n_hi": 8192, "L_lo": 0, "L_hi": 0, "T": 0, "lens": 3},
        # Decoding rows and chunks of prompts in one batch (odd lengths, five query heads to a key head, heads of 64).
        {"name": "mixed_dh64", "op": "attn", "dtype": "bf16", "H": 40, "Hkv": 8, "Dh": 64, "ps": 32, "B": 11,
         "n_lo": 1, "n_hi": 700, "L_lo": 0, "L_hi": 5000, "T": 0, "lens": 4},
        # The 33B batch's verify step: a tree of 65 rows on each of four ragged prefixes, 52 heads.
        {"name": "tree_33b_bs4", "op": "attn", "dtype": "bf16", "H": 52, "Hkv": 52, "Dh": 128, "ps": 16, "B": 4,
         "n_lo": 65, "n_hi": 65, "L_lo": 512, "L_hi": 8192, "T": 65, "lens": 5},
        # float32 chunks: the element type of the framework's exact runs.
        {"name": "chunk_f32", "op": "attn", "dtype": "f32", "H": 16, "Hkv": 4, "Dh": 64, "ps": 16, "B": 5,
         "n_lo": 1, "n_hi": 300, "L_lo": 0, "L_hi": 2000, "T": 0, "lens": 6},
        # A few parallel samples of two prompts.
        {"name": "pages_small", "op": "pages", "dtype": "bf16", "Hkv": 8, "Dh": 128, "ps": 16, "parents": 2, "fan": 3,
         "done": 2, "L_lo": 20, "L_hi": 600, "n_hi": 4, "lens": 7},
        # A full server: 64 prompts with four samples each, 100 rows finished.
        {"name": "pages_large", "op": "pages", "dtype": "bf16", "Hkv": 8, "Dh": 128, "ps": 16, "parents": 64, "fan": 4,
         "done": 100, "L_lo": 100, "L_hi": 4096, "n_hi": 65, "lens": 8},
        # A small pool after a few rows ended.
        {"name": "compact_small", "op": "compact", "dtype": "bf16", "Hkv": 32, "Dh": 128, "ps": 16, "num_pages": 601,
         "live": 300, "moves": 60, "rows": 8},
        # A pool of 4.3 GB, half of it live, a quarter of it out of place.
        {"name": "compact_large", "op": "compact", "dtype": "bf16", "Hkv": 8, "Dh": 128, "ps": 16, "num_pages": 65536,
         "live": 32768, "moves": 16384, "rows": 256},
        # The accepted path of the 7B step.
        {"name": "accept_one", "op": "accept", "dtype": "bf16", "Hkv": 32, "Dh": 128, "ps": 16, "B": 1, "T": 65, "K": 4,
         "L_lo": 1024, "L_hi": 1024, "lens": 9},
        # Sixteen sequences of the 33B shape (the most a verify step takes).
        {"name": "accept_batch16", "op": "accept", "dtype": "bf16", "Hkv": 52, "Dh": 128, "ps": 16, "B": 16, "T": 65,
         "K": 5, "L_lo": 512, "L_hi": 8192, "lens": 10},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "attn", "pages", "compact", "accept"])
    lens = rng.randrange(1 << 30)
    if op == "pages":
        return {"op": op, "dtype": rng.choice(["bf16", "bf16", "f32"]), "Hkv": rng.choice([1, 2, 4, 8]),
                "Dh": rng.choice([64, 128]), "ps": rng.choice([16, 32, 64]), "parents": _log(rng, 1, 64),
                "fan": rng.randint(1, 5), "done": _log(rng, 1, 100), "L_lo": 1, "L_hi": _log(rng, 40, 3000),
                "n_hi": _log(rng, 1, 65), "lens": lens}
    if op == "compact":
        n = _log(rng, 40, 40000)
        live = rng.randint(n // 4, n // 2)
        return {"op": op, "dtype": rng.choice(["bf16", "bf16", "f32"]), "Hkv": rng.choice([1, 2, 5, 8]),
                "Dh": rng.choice([64, 128]), "ps": 16, "num_pages": n, "live": live, "moves": rng.randint(0, live // 2),
                "rows": _log(rng, 1, 256)}
    if op == "accept":
        return {"op": op, "dtype": rng.choice(["bf16", "bf16", "f32"]), "Hkv": rng.choice([1, 3, 8, 32, 52]),
                "Dh": rng.choice([64, 128]), "ps": rng.choice([16, 32, 64, 128]), "B": rng.randint(1, 16),
                "T": rng.randint(20, 300), "K": rng.randint(1, 8), "L_lo": 0, "L_hi": _log(rng, 1, 8192), "lens": lens}
    while True:
        form = rng.choice(["decode", "decode", "chunk", "mixed", "tree"])
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        Hkv, g = rng.choice([1, 2, 4, 8, 13, 32]), rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 16])
        c = {"op": op, "dtype": dtype, "H": Hkv * g, "Hkv": Hkv, "Dh": rng.choice([64, 128]),
             "ps": rng.choice([16, 16, 32, 64, 128, 256]), "B": 1, "n_lo": 1, "n_hi": 1, "L_lo": 0, "L_hi": 0, "T": 0,
             "lens": lens}
        if Hkv * g > 64:
            continue
        if form == "decode":
            c |= {"B": _log(rng, 1, 128), "n_hi": rng.choice([1, 1, 1, 2, 4]), "L_hi": _log(rng, 1, 60000)}
        elif form == "chunk":
            n = _log(rng, 2, 6000)
            c |= {"B": rng.randint(1, 2), "n_lo": n, "n_hi": n, "L_hi": _log(rng, 1, 8192)}
        elif form == "mixed":
            c |= {"B": rng.randint(2, 24), "n_hi": _log(rng, 2, 1200), "L_hi": _log(rng, 1, 8192)}
        else:
            t = rng.randint(2, 257)
            c |= {"B": rng.randint(1, 8), "n_lo": t, "n_hi": t, "T": t, "L_hi": _log(rng, 1, 8192)}
        top = c["L_hi"] + c["n_hi"]
        pairs, slab = c["B"] * c["H"] * c["n_hi"] * top, c["B"] * top * Hkv * c["Dh"]
        if pairs <= 2 ** 31 and slab <= 2 ** 29 and pairs * c["Dh"] <= (2 ** 38 if dtype == "bf16" else 2 ** 32):
            return c


def _lengths(case):
    """New tokens and prefix of every sequence (attn), or the prefixes alone."""
    r = random.Random(case["lens"])
    if case["op"] == "attn":
        n = []
        for b in range(case["B"]):  # about half the rows of a mixed batch decode, the others bring a chunk
            one = case["n_lo"] < case["n_hi"] and r.random() < 0.5
            n.append(case["n_lo"] if one else r.randint(case["n_lo"], case["n_hi"]))
        if case["n_hi"] > case["n_lo"]:
            n[-1] = case["n_hi"]
        return n, [r.randint(case["L_lo"], case["L_hi"]) for _ in n]
    count = case["B"] if case["op"] == "accept" else case["parents"] + case["done"]
    return [r.randint(case["L_lo"], case["L_hi"]) for _ in range(count)]


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    D = case["Dh"]
    if case["op"] == "attn":
        n, L = _lengths(case)
        tokens, keys = sum(n), sum(a + b for a, b in zip(n, L))
        if case["T"]:  # the tree's rows see about depth + 1 of its nodes
            depth = _tree_depth(case["T"])
            pairs = sum(a * b for a, b in zip(n, L)) + len(n) * sum(d + 1 for d in depth)
        else:
            pairs = sum(a * b + a * (a + 1) // 2 for a, b in zip(n, L))
        return {"bytes": e * D * (2 * tokens * case["H"] + 4 * tokens * case["Hkv"] + 2 * keys * case["Hkv"]),
                "flops": 4 * case["H"] * D * pairs}
    if case["op"] == "pages":
        L = _lengths(case)[:case["parents"]]
        lines = sum(case["fan"] * (x % case["ps"]) for x in L)  # one copy of the tail for every child but the last sharer
        pages = sum(-(-x // case["ps"]) for x in L) * (case["fan"] + 1)
        return {"bytes": 4 * lines * case["Hkv"] * D * e + 12 * pages, "flops": 0}
    if case["op"] == "compact":
        return {"bytes": 4 * case["moves"] * case["ps"] * case["Hkv"] * D * e + 8 * case["num_pages"], "flops": 0}
    return {"bytes": 4 * case["B"] * (case["K"] + 1) * case["Hkv"] * D * e, "flops": 0}


# ------------------------------------------------------------------ inputs --

def _tree_parent(T):
    """A breadth-first tree of T rows: node i's parent is (i - 1) / 4."""
    return [-1] + [(i - 1) // 4 for i in range(1, T)]


def _tree_depth(T):
    depth = [0] * T
    for i, p in enumerate(_tree_parent(T)):
        depth[i] = 0 if p < 0 else depth[p] + 1
    return depth


def _views(meta, rows, max_pages, num_pages):
    w = -(-num_pages // 32)
    refs, bits, length, held, table = torch.split(meta, [num_pages, w, rows, rows, rows * max_pages])
    return refs, bits, length, held, table.view(rows, max_pages)


def _bits_of(refs):
    """free_bits of these refs: bit p % 32 of word p / 32 is set where page p is free."""
    n = refs.numel()
    free = torch.zeros(-(-n // 32) * 32, dtype=torch.int64, device=refs.device)
    free[:n] = (refs == 0).long()
    words = (free.view(-1, 32) << torch.arange(32, device=refs.device)).sum(1)
    return torch.where(words >= 2 ** 31, words - 2 ** 32, words).int()


def _cache(gen, lengths, room, ps, Hkv, D, dt, spare, rows, max_pages, num_pages=None):
    """A pool whose rows hold `lengths` tokens in pages taken in random order, with room for `room` more each."""
    dev = "cuda"
    count = [-(-(x + y) // ps) for x, y in zip(lengths, room)]
    num_pages = num_pages or sum(count) + spare
    order = torch.randperm(num_pages, generator=gen, device=dev).int()
    meta = torch.zeros(num_pages + -(-num_pages // 32) + 2 * rows + rows * max_pages, dtype=torch.int32, device=dev)
    refs, bits, length, held, table = _views(meta, rows, max_pages, num_pages)
    table.fill_(-1)
    used = len(lengths)
    length[:used] = torch.tensor(lengths, dtype=torch.int32, device=dev)
    held[:used] = torch.tensor(count, dtype=torch.int32, device=dev)
    mine = torch.arange(max_pages, device=dev)[None] < held[:, None]
    table[mine] = order[:sum(count)]
    refs[order[:sum(count)].long()] = 1
    bits.copy_(_bits_of(refs))
    pool = [torch.randn(num_pages, Hkv, ps, D, generator=gen, device=dev, dtype=dt) for _ in range(2)]
    return meta, pool, num_pages


def prepare(case, seed):
    dev, dt = "cuda", DT[case["dtype"]]
    gen = torch.Generator(device=dev).manual_seed(seed)
    host = random.Random(seed)
    ps, Hkv, D = case["ps"], case["Hkv"], case["Dh"]
    s = {"case": case}
    i32 = {"dtype": torch.int32, "device": dev}
    if case["op"] == "attn":
        n, L = _lengths(case)
        B, H = case["B"], case["H"]
        rows = B + 3  # the batch's rows lie anywhere among the cache's
        where = host.sample(range(rows), B)
        all_l, all_n = [0] * rows, [0] * rows
        for b, r in enumerate(where):
            all_l[r], all_n[r] = L[b], n[b]
        max_pages = max(1, max(-(-(x + y) // ps) for x, y in zip(L, n)))
        s["meta"], pool, s["num_pages"] = _cache(gen, all_l, all_n, ps, Hkv, D, dt, 5, rows, max_pages)
        s["k_pages"], s["v_pages"] = pool
        s |= {"rows": rows, "max_pages": max_pages, "max_new": max(n), "top": max(x + y for x, y in zip(L, n))}
        s["where"] = torch.tensor(where, **i32)
        s["q_start"] = torch.tensor([sum(n[:b]) for b in range(B + 1)], **i32)
        total = sum(n)
        # q, k and v of a token lie side by side, as one projection writes them
        qkv = torch.randn(total, H + 2 * Hkv, D, generator=gen, device=dev, dtype=dt)
        s["q"], s["k_new"], s["v_new"] = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
        s["out"] = torch.zeros(total, H, D, dtype=dt, device=dev)
        s["err"] = torch.zeros(1, **i32)
        s["tree"] = None
        if case["T"]:
            T = case["T"]
            parent, depth = _tree_parent(T), _tree_depth(T)
            anc = torch.zeros(T, T, dtype=torch.bool)
            for i in range(T):
                a = i
                while a >= 0:
                    anc[i, a] = True
                    a = parent[a]
            s["tree"] = {"parent": torch.tensor(parent, dtype=torch.int32), "depth": torch.tensor(depth, **i32),
                         "anc": anc.to(dev)}
    elif case["op"] == "pages":
        P, fan, done = case["parents"], case["fan"], case["done"]
        lengths = _lengths(case)
        rows = P + done + P * fan
        max_pages = -(-(case["L_hi"] + case["n_hi"]) // ps)
        extra = P * fan * (1 + -(-case["n_hi"] // ps)) + P * -(-case["n_hi"] // ps)
        s["saved"], pool, s["num_pages"] = _cache(gen, lengths, [0] * len(lengths), ps, Hkv, D, dt, extra + 7, rows,
                                                  max_pages)
        s["meta"] = s["saved"].clone()
        s["k_pages"], s["v_pages"] = pool
        s |= {"rows": rows, "max_pages": max_pages}
        keep = [-1] * rows
        for r in range(P, P + done):
            keep[r] = 0
        s["keep"] = torch.tensor(keep, **i32)
        child = list(range(P + done, rows))
        host.shuffle(child)
        s["src"] = torch.tensor([p for p in range(P) for _ in range(fan)], **i32)
        s["dst"] = torch.tensor(child, **i32)
        n_new = [host.randint(1, case["n_hi"]) if r < P or r >= P + done else 0 for r in range(rows)]
        s["n_new"] = torch.tensor(n_new, **i32)
        s["copies"] = torch.zeros(rows, 4, **i32)
        s["n_copies"] = torch.zeros(1, **i32)
        s["granted"] = torch.zeros(rows, **i32)
        s["err"] = torch.zeros(1, **i32)
    elif case["op"] == "compact":
        N, live, moves, rows = case["num_pages"], case["live"], case["moves"], case["rows"]
        low = torch.randperm(live, generator=gen, device=dev)[:live - moves]
        high = live + torch.randperm(N - live, generator=gen, device=dev)[:moves]
        pages = torch.cat([low, high])[torch.randperm(live, generator=gen, device=dev)].int()
        each = -(-live // rows)
        max_pages = each + 2
        saved = torch.zeros(N + -(-N // 32) + 2 * rows + rows * max_pages, **i32)
        refs, bits, length, held, table = _views(saved, rows, max_pages, N)
        table.fill_(-1)
        held.copy_((live - torch.arange(rows, device=dev) * each).clamp(0, each).int())
        length.copy_(held * ps)
        mine = torch.arange(max_pages, device=dev)[None] < held[:, None]
        table[mine] = pages
        # every eighth row's first page is shared with the row after it
        pair = torch.arange(0, rows - 1, 8, device=dev)
        pair = pair[(held[pair] < max_pages) & (held[pair + 1] > 0)]
        table[pair, held[pair].long()] = table[pair + 1, 0]
        held[pair] += 1
        length[pair] += ps
        refs.copy_(torch.bincount(table[table >= 0].long(), minlength=N).int())
        bits.copy_(_bits_of(refs))
        s |= {"saved": saved, "meta": saved.clone(), "rows": rows, "max_pages": max_pages, "num_pages": N}
        s["k_pages"] = torch.randn(N, Hkv, ps, D, generator=gen, device=dev, dtype=dt)
        s["v_pages"] = torch.randn(N, Hkv, ps, D, generator=gen, device=dev, dtype=dt)
        s["copies"] = torch.zeros(max(1, moves), 4, **i32)
        s["n_copies"] = torch.zeros(1, **i32)
        s["err"] = torch.zeros(1, **i32)
    else:
        B, T, K = case["B"], case["T"], case["K"]
        lengths = _lengths(case)
        max_pages = max(-(-(x + T) // ps) for x in lengths)
        s["saved"], pool, s["num_pages"] = _cache(gen, lengths, [T] * B, ps, Hkv, D, dt, 3, B, max_pages)
        s["meta"] = s["saved"].clone()
        s["k_pages"], s["v_pages"] = pool
        s |= {"rows": B, "max_pages": max_pages}
        nodes, alen = [], []
        for _ in range(B):  # a path whose first nodes may lie in place, the others past the accepted range
            a = host.randint(0, K)
            first = host.randint(0, a)
            rest = sorted(host.sample(range(K + 1, T), a - first))
            nodes.append(list(range(first + 1)) + rest + [-1] * (K - a))
            alen.append(a)
        s["nodes"], s["accept_len"] = torch.tensor(nodes, **i32), torch.tensor(alen, **i32)
        s["err"] = torch.zeros(1, **i32)
    return s


# ------------------------------------------------------------ the operators --

def run(s):
    if own:
        return _run_own(s)
    return {"attn": _plain_attn, "pages": _plain_pages, "compact": _plain_compact, "accept": _plain_accept}[
        s["case"]["op"]](s)


def _run_own(s):
    from medusa_tree_speculative_gb300 import medusa as M

    case = s["case"]
    if "handle" not in s:  # what a program makes once: the cache's handle, the workspace, the tree
        s["handle"] = M.Pages.from_state(s["meta"], s["rows"], s["max_pages"], s["num_pages"], case["ps"])
        if case["op"] == "attn":
            s["work"] = torch.zeros(M.medusa_paged_attn_workspace_size(
                case["B"], s["q"].shape[0], s["max_new"], case["H"], case["Hkv"], case["Dh"], s["q"].dtype),
                dtype=torch.uint8, device="cuda")
            s["dtree"] = _device_tree(M, s) if s["tree"] else None
        if case["op"] == "compact":
            s["work"] = torch.empty(M.medusa_pages_compact_workspace_size(s["num_pages"]), dtype=torch.uint8,
                                    device="cuda")
    pages = s["handle"]
    if case["op"] == "attn":
        M.medusa_paged_attn(s["q"], s["k_new"], s["v_new"], s["k_pages"], s["v_pages"], pages, s["where"],
                            s["q_start"], s["max_new"], s["dtree"], THETA, 1.0 / math.sqrt(case["Dh"]), s["out"],
                            s["work"], s["err"])
        return {"out": s["out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"], "err": s["err"]}
    s["meta"].copy_(s["saved"])
    if case["op"] == "pages":
        M.medusa_pages_free(pages, s["keep"], s["err"])
        M.medusa_pages_fork(pages, s["src"], s["dst"], s["err"])
        M.medusa_pages_reserve(pages, s["n_new"], s["copies"], s["n_copies"], s["granted"], s["err"])
        M.medusa_pages_copy(s["k_pages"], s["v_pages"], s["copies"], s["n_copies"], s["err"])
        M.medusa_pages_commit(pages, None, s["n_new"], 0, s["err"])
        return {k: s[k] for k in ("meta", "copies", "n_copies", "granted", "k_pages", "v_pages", "err")}
    if case["op"] == "compact":
        M.medusa_pages_compact(pages, s["copies"], s["n_copies"], s["work"], s["err"])
        M.medusa_pages_copy(s["k_pages"], s["v_pages"], s["copies"], s["n_copies"], s["err"])
        return {k: s[k] for k in ("meta", "copies", "n_copies", "k_pages", "v_pages", "err")}
    M.medusa_paged_compact(s["k_pages"], s["v_pages"], pages, None, s["nodes"], s["accept_len"], case["T"], s["err"])
    M.medusa_pages_commit(pages, None, s["accept_len"], 1, s["err"])
    return {k: s[k] for k in ("meta", "k_pages", "v_pages", "err")}


def _device_tree(M, s):
    """The case's tree as the framework compiles it (node i's parent is (i - 1) / 4: rank path by rank path)."""
    parent = s["tree"]["parent"].tolist()
    T, K = len(parent), max(1, int(s["tree"]["depth"].max()))
    paths, plen = torch.zeros(T - 1, K, dtype=torch.int32), []
    for i in range(1, T):
        path, a = [], i
        while a > 0:
            path.append((a - 1) % 4 + 1)
            a = parent[a]
        paths[i - 1, :len(path)] = torch.tensor(path[::-1])
        plen.append(len(path))
    return M.DeviceTree(M.medusa_tree_compile(paths.numpy(), plen, K))


def _rotate(x, pos):
    """x [N][heads][D] in float32, pos [N]: pairs (j, j + D/2) turned by pos * theta^(-2j/D); angles in 64 bits."""
    D = x.shape[-1]
    j = torch.arange(D // 2, device=x.device, dtype=torch.float64)
    ang = pos.double()[:, None] * THETA ** (-2.0 * j / D)
    c, t = ang.cos().float()[:, None], ang.sin().float()[:, None]
    lo, hi = x[..., :D // 2], x[..., D // 2:]
    return torch.cat([lo * c - hi * t, hi * c + lo * t], -1)


def _plain_attn(s):
    case = s["case"]
    H, Hkv, D, ps = case["H"], case["Hkv"], case["Dh"], case["ps"]
    g, B, total, most = H // Hkv, case["B"], s["q"].shape[0], s["max_new"]
    refs, bits, length, held, table = _views(s["meta"], s["rows"], s["max_pages"], s["num_pages"])
    row, start = s["where"].long(), s["q_start"].long()
    L, n = length[row].long(), start[1:] - start[:-1]
    tok = torch.arange(total, device="cuda")
    b = torch.searchsorted(start[1:], tok, right=True)
    i = tok - start[b]
    pos = L[b] + (s["tree"]["depth"].long()[i] if s["tree"] else i)
    q = _rotate(s["q"].float(), pos) / math.sqrt(D)
    slot = L[b] + i
    page, line = table[row[b], slot // ps].long(), slot % ps
    s["k_pages"][page, :, line] = _rotate(s["k_new"].float(), pos).to(s["k_pages"].dtype)
    s["v_pages"][page, :, line] = s["v_new"]
    # every sequence's cache and queries, padded to the longest
    top = s["top"]
    width = -(-top // ps)
    at = table[row, :width].clamp(min=0).long()
    k = s["k_pages"][at].permute(0, 2, 1, 3, 4).reshape(B, Hkv, width * ps, D)[:, :, :top].float()
    v = s["v_pages"][at].permute(0, 2, 1, 3, 4).reshape(B, Hkv, width * ps, D)[:, :, :top].float()
    key = torch.arange(top, device="cuda")
    v = v * (key < (L + n)[:, None])[:, None, :, None]
    pad = torch.zeros(B, most, H, D, device="cuda")
    pad[b, i] = q
    pad = pad.view(B, most, Hkv, g, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, most * g, D)
    score = pad @ k.transpose(-1, -2)
    qi = torch.arange(most, device="cuda")
    if s["tree"]:
        node = key[None] - L[:, None]
        anc = s["tree"]["anc"][:, node.clamp(0, case["T"] - 1)].permute(1, 0, 2)
        seen = (node < 0)[:, None] | (anc & ((node >= 0) & (node < case["T"]))[:, None])
    else:
        seen = key[None, None] <= (L[:, None] + qi[None])[..., None]
    score = score.view(B, Hkv, most, g, top).masked_fill_(~seen[:, None, :, None], -math.inf)
    score -= score.amax(-1, keepdim=True)
    score.exp_()
    total_p = score.sum(-1, keepdim=True)
    o = (score.view(B, Hkv, most * g, top) @ v).view(B, Hkv, most, g, D) / total_p
    s["out"].copy_(o.permute(0, 2, 1, 3, 4).reshape(B, most, H, D)[b, i])
    return {"out": s["out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"], "err": s["err"]}


def _plain_pages(s):
    case, ps = s["case"], s["case"]["ps"]
    s["meta"].copy_(s["saved"])
    refs, bits, length, held, table = _views(s["meta"], s["rows"], s["max_pages"], s["num_pages"])
    col = torch.arange(s["max_pages"], device="cuda")
    N = s["num_pages"]
    # free: pages past the kept length lose a reference
    cut = s["keep"] >= 0
    new_len = torch.where(cut, torch.minimum(length, s["keep"]), length)
    new_held = torch.where(cut, (new_len + ps - 1) // ps, held)
    gone = (col[None] >= new_held[:, None]) & (col[None] < held[:, None])
    refs.index_add_(0, table.clamp(min=0).view(-1).long(), -gone.view(-1).int())
    table.masked_fill_(gone, -1)
    length.copy_(new_len)
    held.copy_(new_held)
    # fork: the child holds the parent's pages
    src, dst = s["src"].long(), s["dst"].long()
    own_pages = (length[src] + ps - 1) // ps
    copied = torch.where(col[None] < own_pages[:, None], table[src], -1)
    table[dst] = copied
    length[dst] = length[src]
    held[dst] = own_pages
    refs.index_add_(0, copied.clamp(min=0).view(-1).long(), (copied >= 0).view(-1).int())
    # reserve: rows in order; a shared tail page is copied, all but its last sharer taking a copy
    rows = torch.arange(s["rows"], device="cuda")
    n = s["n_new"]
    tail = table[rows, (length // ps).clamp(max=s["max_pages"] - 1).long()].clamp(min=0).long()
    partial = (n > 0) & (length % ps != 0)
    same = (tail[:, None] == tail[None]) & partial[:, None] & partial[None] & (rows[None] < rows[:, None])
    cow = partial & (refs[tail] - same.sum(1) > 1)
    more = torch.where(n > 0, ((length + n + ps - 1) // ps - held).clamp(min=0), 0)
    need = more + cow.int()
    upto = need.cumsum(0)
    ok = upto <= (refs == 0).sum()
    s["granted"].copy_(ok.int())
    need, cow, more = need * ok, cow & ok, more * ok
    first = (upto - need).long()
    free = torch.argsort((refs > 0).int(), stable=True)
    lead = free[first.clamp(max=N - 1)]
    spot = cow.int().cumsum(0) - 1
    s["n_copies"].copy_(cow.sum()[None])
    entry = torch.stack([tail.int(), lead.int(), length % ps, rows.int()], 1)
    put = torch.where(cow, spot, s["rows"]).long()  # rows without a copy write a line that is cut off
    lines = torch.cat([s["copies"], s["copies"][:1]])
    lines[put] = entry
    s["copies"].copy_(lines[:-1])
    refs.index_add_(0, tail, -cow.int())
    where_cow = (length // ps).long()[:, None] == col[None]
    grown = (col[None] >= held[:, None]) & (col[None] < (held + more)[:, None])
    nth = first[:, None] + cow.long()[:, None] + (col[None] - held[:, None])
    table.copy_(torch.where(where_cow & cow[:, None], lead.int()[:, None], torch.where(
        grown, free[nth.clamp(0, N - 1)].int(), table)))
    refs.index_add_(0, free, (torch.arange(N, device="cuda") < need.sum()).int())
    held += more
    bits.copy_(_bits_of(refs))
    # the copies: the first lines of each tail page
    c = s["copies"][:s["rows"]]
    live = torch.arange(s["rows"], device="cuda") < s["n_copies"]
    a, z = c[:, 0].long(), torch.where(live, c[:, 1], c[:1, 1]).long()
    lines = (torch.arange(ps, device="cuda")[None] < c[:, 2:3])[:, None, :, None]
    a = torch.where(live, a, a[:1])
    lines = torch.where(live[:, None, None, None], lines, lines[:1])
    any_copy = s["n_copies"] > 0
    for pool in (s["k_pages"], s["v_pages"]):
        pool.index_copy_(0, z, torch.where(lines & any_copy, pool[a], pool[z]))
    length += torch.where(n > 0, n, 0)
    return {k: s[k] for k in ("meta", "copies", "n_copies", "granted", "k_pages", "v_pages", "err")}


def _plain_compact(s):
    s["meta"].copy_(s["saved"])
    refs, bits, length, held, table = _views(s["meta"], s["rows"], s["max_pages"], s["num_pages"])
    N = s["num_pages"]
    page = torch.arange(N, device="cuda")
    live = refs > 0
    count = live.sum()
    out, hole = live & (page >= count), ~live & (page < count)
    moves = out.sum()
    most = s["copies"].shape[0]
    src = torch.argsort((~out).int(), stable=True)[:most]
    dst = torch.argsort((~hole).int(), stable=True)[:most]
    on = torch.arange(most, device="cuda") < moves
    s["n_copies"].copy_(moves[None])
    entry = torch.stack([src, dst, torch.full_like(src, s["case"]["ps"]), torch.full_like(src, -1)], 1).int()
    s["copies"].copy_(torch.where(on[:, None], entry, s["copies"]))
    to = torch.where(on, dst, src)  # lines past the last move copy a page onto itself
    goes = page.clone().index_copy_(0, src, to)
    table.copy_(torch.where(table >= 0, goes[table.clamp(min=0).long()].int(), table))
    moved = refs[src]
    refs.index_copy_(0, src, torch.where(on, 0, moved))
    refs.index_copy_(0, to, moved)
    bits.copy_(_bits_of(refs))
    for pool in (s["k_pages"], s["v_pages"]):
        pool.index_copy_(0, to, pool[src])
    return {k: s[k] for k in ("meta", "copies", "n_copies", "k_pages", "v_pages", "err")}


def _plain_accept(s):
    case, ps = s["case"], s["case"]["ps"]
    s["meta"].copy_(s["saved"])
    refs, bits, length, held, table = _views(s["meta"], s["rows"], s["max_pages"], s["num_pages"])
    j = torch.arange(case["K"] + 1, device="cuda")
    used = j[None] <= s["accept_len"][:, None]
    to = length[:, None] + j[None]
    frm = length[:, None] + torch.where(used, s["nodes"], j[None].int())  # unused lines copy a token onto itself
    row = torch.arange(case["B"], device="cuda")[:, None]
    cols = s["max_pages"] - 1
    fp, tp = table[row, (frm // ps).clamp(max=cols).long()].long(), table[row, (to // ps).clamp(max=cols).long()].long()
    fl, tl = (frm % ps).long(), (to % ps).long()
    for pool in (s["k_pages"], s["v_pages"]):
        pool[tp, :, tl] = pool[fp, :, fl]
    length += s["accept_len"] + 1
    return {k: s[k] for k in ("meta", "k_pages", "v_pages", "err")}


# -------------------------------------------------- the definition, in 64 bits --

def exact(case, seed):
    s = prepare(case, seed)
    return {"attn": _exact_attn, "pages": _exact_pages, "compact": _exact_compact, "accept": _exact_accept}[case["op"]](s)


def _exact_attn(s):
    case = s["case"]
    n, L = _lengths(case)
    H, Hkv, D, ps = case["H"], case["Hkv"], case["Dh"], case["ps"]
    if 4 * H * D * sum(a * (a + b) for a, b in zip(n, L)) > 6e12:
        return None
    refs, bits, length, held, table = _views(s["meta"], s["rows"], s["max_pages"], s["num_pages"])
    kp, vp = s["k_pages"].double(), s["v_pages"].double()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    freq = torch.tensor([THETA ** (-2.0 * j / D) for j in range(D // 2)], dtype=torch.float64, device="cuda")
    at = 0
    for b, r in enumerate(s["where"].tolist()):
        i = torch.arange(n[b], device="cuda")
        pos = (L[b] + (s["tree"]["depth"][i] if s["tree"] else i)).double()
        turn = torch.polar(torch.ones(n[b], D // 2, dtype=torch.float64, device="cuda"), pos[:, None] * freq)

        def rot(x):
            x = x[at:at + n[b]].double()
            z = torch.complex(x[..., :D // 2], x[..., D // 2:]) * turn[:, None]
            return torch.cat([z.real, z.imag], -1)

        q, k, v = rot(s["q"]), rot(s["k_new"]), s["v_new"][at:at + n[b]].double()
        ids = table[r].tolist()
        for t in range(n[b]) if n[b] < 64 else ():
            kp[ids[(L[b] + t) // ps], :, (L[b] + t) % ps] = k[t]
            vp[ids[(L[b] + t) // ps], :, (L[b] + t) % ps] = v[t]
        if n[b] >= 64:
            x = L[b] + i
            kp[table[r].long()[x // ps], :, x % ps] = k
            vp[table[r].long()[x // ps], :, x % ps] = v
        keys = L[b] + n[b]
        x = torch.arange(keys, device="cuda")
        seen = torch.cat([torch.ones(n[b], L[b], dtype=torch.bool, device="cuda"), s["tree"]["anc"]], 1) if s["tree"] \
            else x[None] <= (L[b] + i)[:, None]
        lead = table[r].long()[x // ps]
        for h in range(Hkv):
            # attention reads what the cache holds: keys rounded to its type
            kh, vh = kp[lead, h, x % ps].to(s["k_pages"].dtype).double(), vp[lead, h, x % ps]
            for m in range(h * (H // Hkv), (h + 1) * (H // Hkv)):
                z = (q[:, m] @ kh.T) / math.sqrt(D)
                out[at:at + n[b], m] = torch.softmax(z.masked_fill_(~seen, -math.inf), -1) @ vh
        at += n[b]
    return {"out": out, "k_pages": kp, "v_pages": vp, "err": None}


def _exact_pages(s):
    """Row by row and page by page, on lists."""
    ps = s["case"]["ps"]
    meta = s["saved"].cpu().clone()
    refs, bits, length, held, table = _views(meta, s["rows"], s["max_pages"], s["num_pages"])
    R, ln, hd, tb = refs.tolist(), length.tolist(), held.tolist(), table.tolist()
    for r, keep in enumerate(s["keep"].tolist()):
        if keep >= 0:
            ln[r] = min(ln[r], keep)
            for c in range(-(-ln[r] // ps), hd[r]):
                R[tb[r][c]] -= 1
                tb[r][c] = -1
            hd[r] = -(-ln[r] // ps)
    for a, z in zip(s["src"].tolist(), s["dst"].tolist()):
        ln[z], hd[z] = ln[a], -(-ln[a] // ps)
        for c in range(hd[z]):
            tb[z][c] = tb[a][c]
            R[tb[a][c]] += 1
    free = [p for p, x in enumerate(R) if x == 0]
    copies, granted, taken, short = [], [], 0, False
    for r, n in enumerate(s["n_new"].tolist()):
        if n == 0:
            granted.append(0 if short else 1)
            continue
        t = ln[r] // ps
        cow = ln[r] % ps != 0 and R[tb[r][t]] > 1
        more = max(0, -(-(ln[r] + n) // ps) - hd[r])
        short = short or taken + more + cow > len(free)
        granted.append(0 if short else 1)
        if short:
            continue
        new = free[taken:taken + more + cow]
        taken += len(new)
        if cow:
            R[tb[r][t]] -= 1
            copies.append([tb[r][t], new[0], ln[r] % ps, r])
            tb[r][t] = new[0]
        for c, p in enumerate(new[1 if cow else 0:]):
            tb[r][hd[r] + c] = p
        hd[r] += more
        for p in new:
            R[p] = 1
    for r, n in enumerate(s["n_new"].tolist()):
        ln[r] += max(n, 0)
    for view, values in ((refs, R), (length, ln), (held, hd), (table, tb)):
        view.copy_(torch.tensor(values, dtype=torch.int32))
    bits.zero_()
    for p, x in enumerate(R):
        if x == 0:
            word = int(bits[p // 32]) & 0xFFFFFFFF | 1 << (p % 32)
            bits[p // 32] = word - 2 ** 32 if word >= 2 ** 31 else word
    kp, vp = s["k_pages"].double(), s["v_pages"].double()
    for a, z, m, _ in copies:
        kp[z, :, :m], vp[z, :, :m] = kp[a, :, :m], vp[a, :, :m]
    lines = torch.zeros(s["rows"], 4, dtype=torch.int32)
    if copies:
        lines[:len(copies)] = torch.tensor(copies, dtype=torch.int32)
    return {"meta": meta, "copies": lines, "n_copies": torch.tensor([len(copies)], dtype=torch.int32),
            "granted": torch.tensor(granted, dtype=torch.int32), "k_pages": kp, "v_pages": vp, "err": None}


def _exact_compact(s):
    meta = s["saved"].cpu().clone()
    refs, bits, length, held, table = _views(meta, s["rows"], s["max_pages"], s["num_pages"])
    R = refs.tolist()
    count = sum(x > 0 for x in R)
    out = [p for p in range(count, len(R)) if R[p] > 0]
    hole = [p for p in range(count) if R[p] == 0]
    goes = dict(zip(out, hole))
    for a, z in goes.items():
        R[z], R[a] = R[a], 0
    table.copy_(torch.tensor([[goes.get(p, p) for p in row] for row in table.tolist()], dtype=torch.int32))
    refs.copy_(torch.tensor(R, dtype=torch.int32))
    words = [0] * bits.numel()
    for p, x in enumerate(R):
        words[p // 32] |= (x == 0) << (p % 32)
    bits.copy_(torch.tensor([w - 2 ** 32 if w >= 2 ** 31 else w for w in words], dtype=torch.int32))
    kp, vp = s["k_pages"].double(), s["v_pages"].double()
    for a, z in goes.items():
        kp[z], vp[z] = kp[a], vp[a]
    lines = torch.zeros_like(s["copies"]).cpu()
    if goes:
        lines[:len(out)] = torch.tensor([[a, z, s["case"]["ps"], -1] for a, z in goes.items()], dtype=torch.int32)
    return {"meta": meta, "copies": lines, "n_copies": torch.tensor([len(out)], dtype=torch.int32), "k_pages": kp,
            "v_pages": vp, "err": None}


def _exact_accept(s):
    ps = s["case"]["ps"]
    meta = s["saved"].cpu().clone()
    refs, bits, length, held, table = _views(meta, s["rows"], s["max_pages"], s["num_pages"])
    pools = [s["k_pages"].double(), s["v_pages"].double()]
    for r, (a, nodes) in enumerate(zip(s["accept_len"].tolist(), s["nodes"].tolist())):
        L, ids = int(length[r]), table[r].tolist()
        for pool in pools:
            held_rows = [pool[ids[(L + x) // ps], :, (L + x) % ps].clone() for x in nodes[:a + 1]]
            for j, line in enumerate(held_rows):
                pool[ids[(L + j) // ps], :, (L + j) % ps] = line
        length[r] += a + 1
    return {"meta": meta, "k_pages": pools[0], "v_pages": pools[1], "err": None}
