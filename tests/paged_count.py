"""Inputs for the paged attention in which every key counts: its result is a table of how many keys of each group were
seen, known exactly.  With Gaussian data and thousands of keys the result is small beside the worst case of its
roundings, so that a lost tile may go unseen; here a group of sixteen keys that is lost, doubled or taken from another
place moves its column by a sixteenth of the keys that share it.

"even": all queries are zero, so all scores are equal; key x's value is a one in column (x / 16) mod D.  Scores and
weights are exact in any type, sums are whole numbers: the result is a quotient, rounded.
"needles": in every whole group of sixteen prefix keys one, at a place of its own, has a score far above the others'
(which are zero), the same in all groups, and a value with a one in its group's column; all other values are noise of
weight e^-40.  A key read from a wrong line, page or tile loses its needle."""
import math

import torch

GROUP = 16


def column(x, D):
    return (x // GROUP) % D


def shares(seen, D, used=None):
    """The result for seen [n][X]: the share of the keys used (None: all) that each column has, [n][D] float64."""
    x = torch.arange(seen.shape[1], device=seen.device)
    w = seen.double() if used is None else (seen & used).double()
    w = torch.where(w.sum(1, keepdim=True) > 0, w, seen.double())  # no needle seen: all scores are equal
    one = torch.zeros(len(x), D, dtype=torch.float64, device=seen.device)
    one[x, column(x, D)] = 1.0
    return w @ one / w.sum(1, keepdim=True)


def needles(L, seed):
    """Whether key x of a prefix of L is a needle."""
    g = torch.Generator().manual_seed(seed)
    at = torch.arange(0, L - L % GROUP, GROUP) + torch.randint(0, GROUP, (L // GROUP,), generator=g)
    used = torch.zeros(L, dtype=torch.bool)
    used[at] = True
    return used


def worst(got, want, dtype):
    """The largest error over its bound: one rounding to the type; sum, quotient and product in 32 bits; weights that
    are not quite zero."""
    u = torch.finfo(dtype).eps / 2
    tol = (u + 2.0 ** -22) * want + 1e-9
    return ((got.double() - want).abs() / tol).nan_to_num(nan=math.inf).max().item()
