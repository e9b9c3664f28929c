"""Sampling with the number 0: the first kept token, however little it weighs."""
import numpy as np
import pytest
import torch

from test_gpu_sample import Call, M, logits, plain  # noqa: F401 (M is a fixture)

pytestmark = pytest.mark.gpu


def first(z, t, k, p, m):
    """(token, kept, logp) for u = 0: of the kept tokens the first one whose weight is not 0 in 64 bits."""
    token, kept, logp = plain(z, t, k, p, m, 0.0)
    order = np.argsort(-z.astype(np.float64), kind="stable")
    gap = (z.astype(np.float64) - z[order[0]].astype(np.float64)) / t
    ids = np.sort(order[:kept])
    ids = ids[np.exp(gap[ids]) > 0]
    return int(ids[0]), kept, float(logp - gap[token] + gap[ids[0]])


def check(c):
    z = c.z.cpu().numpy()
    for r in range(z.shape[0]):
        t, k, p, m = (x[r].item() for x in (c.t, c.k, c.p, c.m))
        want = first(z[r], t, k, p, m)
        got = c.token[r].item(), c.kept[r].item(), c.logp[r].item()
        assert got[:2] == want[:2], (r, t, k, p, m, got, want)
        # as Call.check
        assert abs(got[2] - want[2]) <= 2.0 ** -24 * abs(want[2]) + 2.0 ** -28, (r, got, want)
    assert int(c.err.item()) == 0


@pytest.mark.parametrize("V", [2, 50, 4096, 5000, 20000, 40000, 128257, 262144])
@pytest.mark.parametrize("gap", [20.0, 35.0, 60.0, 300.0, 745.0])
def test_the_first_token_weighs_little(M, V, gap):
    """Rows whose first token, whose first half, or whose tokens but the last lie `gap` below the largest one, without
    cuts, with top-k and with min-p that reaches the token or does not."""
    z = torch.zeros(6, V, device="cuda")
    z[0, 0], z[1, :V // 2], z[2, :-1] = -gap, -gap, -gap
    z[3:] = z[:3]
    low = float(np.float32(np.exp(-gap)))
    check(Call(M, z, u=0.0).run())
    check(Call(M, z, k=[V, max(1, V - 1), max(2, V // 2 + 1)] * 2, u=0.0).run())
    check(Call(M, z, m=[low / 2] * 3 + [min(1.0, low * 2)] * 3, u=0.0).run())
    check(Call(M, z * 0.5, t=0.5, u=0.0).run())


@pytest.mark.parametrize("V", [50, 9000, 128257])
def test_weights_that_64_bits_do_not_hold(M, V):
    """They are not drawn, though they are kept."""
    z = torch.zeros(4, V, device="cuda")
    z[0, :3], z[1, 0], z[1, 1], z[2, :V - 1], z[3, 5] = -746.0, -800.0, -745.0, -1e30, 3e38
    check(Call(M, z, u=0.0).run())
    check(Call(M, z, k=V - 1, u=0.0).run())


@pytest.mark.parametrize("V", [300, 20000, 128257])
def test_ordinary_rows(M, V):
    """With top-p no kept token weighs too little to be counted."""
    z = logits(12, V, seed=3)
    check(Call(M, z, t=0.7, p=[0.0, 0.3, 0.9, 1 - 2.0 ** -24] * 3, u=0.0).run())
    check(Call(M, z, t=0.2, k=[0, 40, 1000, 5000] * 3, p=[1 - 2.0 ** -24] * 6 + [0.5] * 6, m=1e-9, u=0.0).run())
    check(Call(M, z, t=3.0, k=[0, 40, 1000, 5000] * 3, m=[0.0, 1e-9, 0.01] * 4, u=0.0).run())


def test_beside_other_numbers(M):
    """Each row by its own number."""
    z = torch.zeros(4, 5000, device="cuda")
    z[:, :4999] = -40.0
    c = Call(M, z, u=[0.0, 0.5, 0.0, 1 - 2.0 ** -24]).run()
    assert c.token.tolist() == [0, 4999, 0, 4999] and c.kept.tolist() == [5000] * 4
