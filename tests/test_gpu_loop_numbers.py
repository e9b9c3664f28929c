"""A decode loop's numbers for its sampled roots serve one step each: a step without new ones says so."""
import pytest
import torch

from medusa_tree_speculative_gb300 import workloads
from test_gpu_paged import M  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu
TOKEN = 1


def make(M, page_size):
    from medusa_tree_speculative_gb300 import loop, step

    w = workloads.get("tiny_fp32")
    t = M.DeviceTree(step.build_tree(w))
    return loop.DecodeLoop(w, loop.StandInModel(w, seed=3), t, 4, L0=w["L"][0], x0=[5] * w["B"], page_size=page_size,
                           sample={"temperature": 0.5})


@pytest.mark.parametrize("page_size", [None, 16])
def test_a_step_without_numbers(M, page_size):
    a = make(M, page_size)
    a.step()
    assert a.st.err.item() == TOKEN and (a.st.next_root == -1).all()


@pytest.mark.parametrize("page_size", [None, 16])
@pytest.mark.parametrize("how", ["argument", "buffer"])
def test_numbers_serve_one_step(M, page_size, how):
    a = make(M, page_size)
    u = torch.full((a.B,), 0.4, device="cuda")
    for _ in range(2):
        if how == "argument":
            a.step(uniforms=u)
        else:
            a.x["uniforms"].copy_(u)
            a.step()
        assert a.st.err.item() == 0 and (a.st.next_root >= 0).all()
    a.step()
    assert a.st.err.item() == TOKEN and (u == 0.4).all()


def test_captured_steps(M):
    a = make(M, 16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        a.step(s)
    for _ in range(2):
        a.x["uniforms"].fill_(0.4)
        g.replay()
        assert a.st.err.item() == 0
    g.replay()
    assert a.st.err.item() == TOKEN
