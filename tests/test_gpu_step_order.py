"""Calls of a step whose inputs are written by the kernel just before them on the stream (the kernels of a call may
start while that one is still running)."""
import pytest
import torch

from quantized_paged_kv_gb300 import workloads as W
from tests import harness as H
from tests.test_gpu_prefix import _Call, _share

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    H.ensure_built()


@pytest.mark.parametrize("splits", [0, 2])
def test_a_plan_put_in_place_by_another_kernel(splits):
    """Two sets of lengths take turns in one plan buffer, each plan written there by a torch kernel."""
    lens = [[1500, 40, 900, 16], [64, 1400, 20, 1000]]
    wl = _share(W.make("tiny_int8", lens=("list", [1500, 1400, 1000, 1000]), seed=95), [0, 4], [16])
    c = _Call(wl, "int8", [0, 4], [16], splits=splits)
    sl = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in lens]
    plans, want = [], []
    for x in sl:
        c.sl = x
        c.launch(checked=True)
        plans.append(c.plan.plan.clone())
        want.append((c.out.clone(), c.lse.clone()))
    assert not torch.equal(plans[0], plans[1])
    for k in range(100):
        c.sl = sl[k % 2]
        torch.add(plans[k % 2], 0, out=c.plan.plan)
        c.launch(update=False)
        torch.cuda.synchronize()
        assert torch.equal(c.out, want[k % 2][0]) and torch.equal(c.lse, want[k % 2][1])


def test_lists_that_run_past_the_plan_are_flagged():
    """The last CTA's list spoiled by more than the plan holds, but less than the prefixes' partial slots: flagged, and
    nothing behind the plan is read."""
    from quantized_paged_kv_gb300 import KvqError

    wl = _share(W.make("tiny_int8", lens=("list", [700, 340, 400]), seed=97), [0, 3], [320])
    c = _Call(wl, "int8", [0, 3], [320], splits=40)
    c.plan.update(c.sl)
    good = c.plan.plan.clone()
    C, A = c.plan.num_ctas, (wl.B + 2 + 3) // 4 * 4
    c.plan.plan[A + 5 * C] += 3 * 40  # o[C]
    with pytest.raises(KvqError):
        c.launch(checked=True, update=False)
    c.plan.plan.copy_(good)
    c.launch(checked=True, update=False)
    c.check()
