"""The checks of test_gpu_paged_every_key see what they are made to see: a result with keys lost, doubled or misplaced
is rejected at every length used there (no GPU needed)."""
import pytest
import torch

from paged_count import needles, shares, worst


def faults(L, n):
    """Name -> the keys seen, as a count each, where something went wrong."""
    X = L + n
    tile = 64
    out = {"zeros": None}

    def lost(name, a, z):
        w = torch.ones(X)
        w[max(0, a):z] = 0
        if w.sum():
            out[name] = w

    lost("first tile", 0, tile)
    lost("last tile", (X - 1) // tile * tile, X)
    mid = X // 2 // tile * tile
    lost("a tile in the middle", mid, mid + tile)
    lost("a page of sixteen", mid, mid + 16)
    lost("one CTA's share", X // 3, X // 2 + 1)
    lost("a quarter", X - X // 4 - 1, X)
    out["a tile twice"] = torch.ones(X)
    out["a tile twice"][mid:mid + tile] = 2
    swapped = torch.ones(X)  # a page read in another one's place
    swapped[mid:mid + 16] = 2
    if mid >= 16:
        swapped[mid - 16:mid] = 0
        out["a page for another"] = swapped
    return out


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("form", ["even", "needles"])
@pytest.mark.parametrize("D,L,n", [(128, 65, 1), (128, 700, 1), (64, 2500, 1), (128, 4000, 1), (64, 4000, 1), (128, 5000, 2),
                                   (64, 9000, 2), (128, 30000, 1), (64, 100001, 3), (128, 100001, 1)])
def test_faults_are_seen(dtype, form, D, L, n):
    seen = torch.ones(1, L + n, dtype=torch.bool)
    used = torch.cat([needles(L, 7), torch.zeros(n, dtype=torch.bool)]) if form == "needles" else None
    want = shares(seen, D, used)
    assert worst(want.to(dtype), want, dtype) <= 1.0
    one = torch.zeros(L + n, D, dtype=torch.float64)
    one[torch.arange(L + n), (torch.arange(L + n) // 16) % D] = 1.0
    for name, w in faults(L, n).items():
        if w is None:
            got = torch.zeros_like(want)
        else:
            w = w.double() * (used.double() if used is not None else 1.0)
            if used is not None and torch.equal(w / w.max(), used.double()):
                continue  # none of the needles, or all of them: their shares are as they were
            got = (w @ one / w.sum())[None]
        assert worst(got.to(dtype), want, dtype) > 1.0, name


def test_needles_lie_in_every_whole_group():
    for L in (0, 1, 15, 16, 17, 1000):
        u = needles(L, 3)
        assert u.numel() == L and int(u.sum()) == L // 16
        assert (u[:L - L % 16].view(-1, 16).sum(1) == 1).all()
