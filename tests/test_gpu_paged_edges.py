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
