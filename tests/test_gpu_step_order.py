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


def test_nothing_shared_without_groups():
    """An empty kvq_prefix with splits = 0: the plan without a prefix, and the decode's result."""
    from quantized_paged_kv_gb300 import DevicePlan, _binding as B, decode

    wl = W.make("tiny_int8", lens=("list", [700, 40, 0, 16]), seed=98)
    cache = H.gpu_cache(wl, "int8")
    sl, bt = torch.from_numpy(wl.seq_lens).cuda(), torch.from_numpy(wl.block_tables).cuda()
    q = torch.from_numpy(wl.q()).to(torch.bfloat16).cuda()
    plan = DevicePlan(cache, wl.B, wl.Hq, bt.shape[1])
    plan.update(sl, checked=True)
    want, out = torch.empty(wl.B, wl.Hq, wl.D, device="cuda"), torch.empty(wl.B, wl.Hq, wl.D, device="cuda")
    lse = torch.empty(wl.B, wl.Hq, device="cuda")
    decode(cache, plan, q, bt, sl, want, wl.sm_scale, checked=True)
    empty = B.KvqPrefixStruct(None, None, 0, 0)
    again = plan.plan.clone().fill_(-9)
    B.kvq_plan_splits_device(cache.struct, sl, 1, bt.shape[1], empty, plan.total_splits, plan.num_ctas, again,
                             plan.workspace, B.KVQ_CHECKED)
    assert torch.equal(again, plan.plan)
    B.kvq_paged_prefix_attention(cache.struct, q, wl.sm_scale, bt, sl, empty, again, plan.total_splits, plan.num_ctas,
                                 plan.workspace, out, lse, B.KVQ_CHECKED)
    assert (out - want).abs().max() <= 4e-3  # each within 2e-3 of the oracle
    assert torch.equal(torch.isneginf(lse), (sl == 0)[:, None].expand_as(lse))


def test_two_steps_at_once():
    """Two streams, each with its own tables, plan and workspaces, over one pool: the same bits as one after the other."""
    from quantized_paged_kv_gb300 import StepTables, build_tables

    calls, tables, want = [], [], []
    for k, (fmt, T, out_dtype) in enumerate((("int8", 1, "f32"), ("int8", 3, "bf16"))):
        wl = _share(W.make("tiny_int8", lens=("list", [1200, 900, 1000, 40, 1300]), seed=110), [0, 5], [640])
        c = _Call(wl, fmt, [0, 5], [640], T=T, splits=3, out_dtype=out_dtype)
        c.cache = calls[0].cache if calls else c.cache
        c.launch(checked=True)
        calls.append(c)
        want.append((c.out.clone(), c.lse.clone()))
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
        t = StepTables(torch.full((300, 40), -1, dtype=torch.int32, device="cuda"), 300 * 200)
        args = i32([3 * k] * 300), i32([100 + (7 * b + k) % 300 for b in range(300)]), i32(list(range(k, 6000 + k)))
        cache = type("Pool", (), {"struct": c.cache.struct})
        build_tables(cache, t, *args, i32([0]))
        tables.append((t, args, t.slot_mapping.clone()))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(50):
        for c, (t, args, _), s in zip(calls, tables, streams):
            with torch.cuda.stream(s):
                c.out.fill_(float("nan"))
                t.slot_mapping.fill_(-7)
                t.free_head.zero_()
                build_tables(type("Pool", (), {"struct": c.cache.struct}), t, *args)
                c.launch()
    torch.cuda.synchronize()
    for c, (t, _, slots), (out, lse) in zip(calls, tables, want):
        assert torch.equal(c.out, out) and torch.equal(c.lse, lse) and torch.equal(t.slot_mapping, slots)
