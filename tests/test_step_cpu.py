"""The step operators without a GPU: the oracle's bookkeeping against examples worked
by hand and against its invariants, the sizes of device plans, and the refusals of the
C entries (made before any CUDA call)."""
import ctypes
import random

import pytest

from oracle import step as ostep
from tests import harness as H


@pytest.fixture(scope="module")
def kvq():
    H.ensure_built()
    import quantized_paged_kv_gb300 as k
    return k


# ------------------------------------------------------------------ the oracle
def test_tables_of_a_worked_example():
    """Pages of 16.  Request 0: 14 tokens + 4: positions 14, 15 on its page 3, 16, 17 on the first free page taken
    (head 1: page 8).  Request 1: nothing to add.  Request 2: 32 tokens (its second page is full) + 1: page 6."""
    got = ostep.build_tables([14, 5, 32], [4, 0, 1], [9, 8, 6, 7], 1, [[3, -1, -1], [4, -1, -1], [1, 2, -1]], 7, 20)
    assert got["block_tables"] == [[3, 8, -1], [4, -1, -1], [1, 2, 6]]
    assert got["slots"] == [3 * 16 + 14, 3 * 16 + 15, 8 * 16, 8 * 16 + 1, 6 * 16, -1, -1]
    assert (got["seq_lens"], got["query_start"], got["page_start"]) == ([18, 5, 33], [0, 4, 4, 5], [0, 1, 1, 2])
    assert got["head"] == 3 and got["bits"] == 0


def test_tables_flag_what_does_not_fit():
    got = ostep.build_tables([0, 40], [20, 9], [5], 0, [[-1, -1, -1], [0, 1, 2]], 29, 4)
    # one free page for two, and its id 5 lies outside a pool of 4; request 1 would run past its 3 pages
    assert got["block_tables"][0] == [5, -1, -1] and got["seq_lens"] == [20, 40]
    assert got["slots"] == [-1] * 29
    assert got["bits"] == ostep.NO_PAGE | ostep.BAD_PAGE | ostep.BAD_SEQLEN
    assert ostep.build_tables([0], [3], [1], 0, [[-1]], 2, 4)["bits"] == ostep.BAD_SLOT


def test_plan_of_a_worked_example():
    """Own pages 5, 2 and 0; 5 splits.  x = 2 gives 3 + 1 + 1 = 5.  Split sizes 1, 2, 2 | 2 | 0; two CTAs take them
    longest first, there and back: (v0 s1), (v0 s2) | (v1), (v0 s0)... in rounds of two."""
    got = ostep.plan([80, 30, 0], 1, 10, 5, 0, [], [], 1, 2)
    assert got[:5] == [0, 3, 4, 5, 2] and got[5:8] == [0, 0, 0]  # offsets, C, padding to a multiple of four
    one = lambda b, s, p, n, direct=0: [b, s, p, n | direct << 23]
    # order: v0 s1 (2 pages), v0 s2 (2), v1 (2), v0 s0 (1), v2 (0): round 0 to CTAs 0, 1, round 1 to 1, 0, round 2 to 0
    assert got[8:16] == one(0, 1, 1, 2) + one(0, 2, 3, 2)
    assert got[16:19] == [0, 2, 3]  # CTA 0 has two more, CTA 1 one
    assert got[20:] == one(0, 0, 0, 1) + one(2, 4, 0, 0, 1) + one(1, 3, 0, 2, 1)


def test_plan_with_a_prefix_of_a_worked_example():
    """Sequences 0 and 1 share 2 pages (35 tokens: two whole pages); slots 0, 1 | 3, 4 are their prefix partials."""
    got = ostep.plan([40, 64, 16], 1, 4, 3 + 3 * 2, 2, [0, 2], [35], 1, 3)
    assert got[:5] == [0, 3, 6, 7, 3]
    d = [got[8 + 4 * i:12 + 4 * i] for i in range(3)]
    assert d == [[1, 5, 2, 2], [0, 2, 2, 1], [2, 6, 0, 1 | 1 << 23]]  # own pages start behind the shared ones


def _items(plan, V, C, n):
    A = (V + 2 + 3) // 4 * 4
    R = (A + 5 * C + 1 + 3) // 4 * 4
    ro = plan[A + 4 * C:A + 5 * C + 1]
    lists = [[plan[A + 4 * c:A + 4 * c + 4]] + [plan[R + 4 * i:R + 4 * i + 4] for i in range(ro[c], ro[c + 1])]
             for c in range(C)]
    assert sum(map(len, lists)) == n and len(plan) == R + 4 * (n - C)
    return lists


def test_plans_cover_every_own_page_once():
    r = random.Random(2)
    for _ in range(60):
        B, q, nhg = r.choice([1, 2, 7, 40]), r.choice([1, 1, 3]), r.choice([1, 2])
        lens = [r.randrange(0, 3000) for _ in range(B)]
        offs = sorted(r.randrange(0, B + 1) for _ in range(3))
        pl = [r.randrange(0, 1500) for _ in range(2)]
        sp = r.choice([1, 4])
        V = B * q
        T = V + r.randrange(0, 90)
        C = r.randrange(1, min(20, T * nhg) + 1)
        plan = ostep.plan(lens, q, 200, T + V * sp, sp, offs, pl, nhg, C)
        seen, loads = {}, []
        for l in _items(plan, V, C, T * nhg):
            for b, split, p0, w in l:
                for p in range(p0, p0 + (w & 0x7FFFFF)):
                    key = (b, w >> 24, p)
                    assert key not in seen
                    seen[key] = split
            loads.append(sum(d[3] & 0x7FFFFF for d in l))
        for b in range(V):
            vis = max(0, lens[b // q] - q + 1 + b % q)
            k = ostep.shared_pages(b // q, offs, pl, 200)
            want = range(k, max(k, -(-vis // 16)))
            for g in range(nhg):
                assert [p for p in range(200) if (b, g, p) in seen] == list(want)
                slots = [seen[b, g, p] for p in want]
                assert slots == sorted(slots)
                assert all(plan[b] + (sp if k else 0) <= s < plan[b + 1] for s in slots)
        assert max(loads) - min(loads) <= max(1, max(max(0, -(-x // 16)) for x in lens))


# ------------------------------------------------------------------ sizes
def _struct(kvq, fmt="int8", pages=4096, hkv=4, d=256):
    return kvq._binding.KvqCacheStruct(None, None, None, None, pages, 16, hkv, d, kvq._binding.FORMATS[fmt], 1.0, 1.0)


@pytest.mark.parametrize("batch,q_len,width,shape,T", [
    (1, 1, 2048, ("int8", 4, 256), 152),        # one wave for one sequence
    (1, 1, 3, ("int8", 4, 256), 3),             # never more splits than pages
    (76, 1, 100, ("int8", 4, 256), 152),        # half a wave of sequences: still one
    (77, 1, 100, ("int8", 4, 256), 304),        # more: a wave more than they fill
    (64, 1, 512, ("int8", 8, 128), 152),        # two head groups a split: (1 + 1) x 152 / 2
    (256, 6, 320, ("int8", 4, 256), 1824),      # 1,536 launch sequences: 12 waves
])
def test_device_plan_sizes(kvq, batch, q_len, width, shape, T):
    s = _struct(kvq, shape[0], hkv=shape[1], d=shape[2])
    nhg = 2 if shape[1] == 8 else 1
    total, ctas, entries = kvq.kvq_plan_device_sizes(s, batch, q_len, width, 0, 152)
    assert (total, ctas) == (T, min(152, T * nhg))
    V = batch * q_len
    A = (V + 2 + 3) // 4 * 4
    assert entries == (A + 5 * ctas + 1 + 3) // 4 * 4 + 4 * (T * nhg - ctas)
    assert kvq.kvq_plan_device_sizes(s, batch, q_len, width, 5, 152) == (T + 5 * V, ctas, entries)


def test_device_plan_sizes_refusals(kvq):
    s = _struct(kvq)
    for args, code in (((0, 1, 10), 1), ((1, 0, 10), 1), ((1, 1, 0), 1), ((4097, 1, 10), 2), ((1025, 4, 10), 2),
                       ((1, 1, 1 << 21), 2), ((4096, 1, (1 << 19) - 1), 2), ((1, 1, 10, -1), 1), ((1, 1, 10, 65), 1),
                       ((1, 1, 10, 0, -1), 1)):
        with pytest.raises(kvq.KvqError) as e:
            kvq.kvq_plan_device_sizes(s, *args[:3], args[3] if len(args) > 3 else 0, args[4] if len(args) > 4 else 152)
        assert e.value.code == code, args
    # the largest widths that the 32-bit sort keys hold
    assert kvq.kvq_plan_device_sizes(s, 4096, 1, (1 << 19) - 2, 0, 152)[0] >= 4096
    assert kvq.kvq_plan_device_sizes(s, 1, 1, (1 << 21) - 1, 0, 152)[0] == 152


def test_prefix_splits_fill_the_device(kvq):
    s = _struct(kvq, hkv=4)
    f = kvq.kvq_prefix_splits
    # 32 sequences x 6 heads = 192 rows: two row blocks x 4 heads = 8 items, 19 key ranges make one wave of 152
    assert f(s, 32, 1, 24, 1, 32768, 152) == 19
    assert 1 <= f(s, 64, 1, 24, 1, 10 ** 6, 152) <= 64
    # few sequences or a short prefix: nothing to share
    assert f(s, 32, 1, 24, 1, 63, 152) == 0 and f(s, 1, 1, 24, 1, 10 ** 6, 152) == 0 and f(s, 4, 1, 24, 1, 0, 152) == 0
    assert f(s, 4, 1, 24, 1, 8192, 152) == 0 < f(s, 4, 1, 24, 1, 32768, 152)
    assert f(s, 16, 1, 24, 1, 2048, 152) == 0 < f(s, 16, 1, 24, 1, 4096, 152)
    for bad in ((0, 1, 24, 1, 64, 0), (4, 0, 24, 1, 64, 0), (4, 1, 23, 1, 64, 0), (4, 1, 24, 5, 64, 0),
                (4, 1, 24, 0, 64, 0), (4, 1, 24, 1, -1, 0)):
        with pytest.raises(kvq.KvqError):
            f(s, *bad)
    with pytest.raises(kvq.KvqError) as e:
        f(_struct(kvq, "int8_g32"), 4, 1, 24, 1, 64, 152)
    assert e.value.code == 2


# ------------------------------------------------------------------ refusals before any CUDA call
P = 1 << 20  # an address that no refused call reads


def _tables(kvq, **over):
    a = dict(cache=_struct(kvq), ctx=P, new=P, batch=4, free=P, num_free=8, head=P, bt=P, width=10, slots=P,
             num_slots=64, sl=P, qs=P, ps=P, head_out=P, ws=P, flags=0)
    a.update(over)
    return kvq.lib().kvq_build_tables(ctypes.byref(a["cache"]), a["ctx"], a["new"], a["batch"], a["free"], a["num_free"],
                                      a["head"], a["bt"], a["width"], a["slots"], a["num_slots"], a["sl"], a["qs"],
                                      a["ps"], a["head_out"], a["ws"], a["flags"], None)


def test_build_tables_refusals(kvq):
    for over, code in (({"batch": 0}, 1), ({"batch": 16385}, 2), ({"width": 0}, 1), ({"num_free": -1}, 1),
                       ({"num_slots": -1}, 1), ({"num_slots": (1 << 40) + 1}, 2), ({"batch": 4096, "width": 1 << 15}, 2),
                       ({"slots": P + 8}, 1), ({"ws": P + 4}, 1), ({"flags": 2}, 1), ({"flags": 8}, 1),
                       ({"free": None}, 1), ({"slots": None}, 1)):
        assert _tables(kvq, **over) == code, over
        assert kvq.kvq_last_error()
    for name in ("ctx", "new", "head", "bt", "sl", "qs", "ps", "head_out", "ws"):
        assert _tables(kvq, **{name: None}) == 1, name
    bad = _struct(kvq)
    bad.page_size = 32
    assert _tables(kvq, cache=bad) == 2


def _prefix(kvq, offs=P, lens=P, groups=1, splits=2):
    return kvq._binding.KvqPrefixStruct(offs, lens, groups, splits)


def _plan(kvq, **over):
    a = dict(cache=_struct(kvq), sl=P, batch=4, q_len=1, width=20, prefix=None, total=152, ctas=152, plan=P, cap=10 ** 6,
             status=P, flags=0)
    a.update(over)
    return kvq.lib().kvq_plan_splits_device(
        ctypes.byref(a["cache"]), a["sl"], a["batch"], a["q_len"], a["width"],
        None if a["prefix"] is None else ctypes.byref(a["prefix"]), a["total"], a["ctas"], a["plan"], a["cap"],
        a["status"], a["flags"], None)


def test_plan_device_refusals(kvq):
    for over, code in (({"sl": None}, 1), ({"plan": None}, 1), ({"status": None}, 1), ({"plan": P + 4}, 1),
                       ({"flags": 4}, 1), ({"flags": 16}, 1), ({"flags": 16, "prefix": _prefix(kvq, splits=0)}, 1),
                       ({"total": 3}, 1), ({"total": 40000}, 1), ({"ctas": 0}, 1), ({"ctas": 153}, 1),
                       ({"cap": 100}, 3), ({"batch": 4097}, 2), ({"q_len": 0}, 1), ({"width": 0}, 1),
                       ({"prefix": _prefix(kvq, offs=None)}, 1), ({"prefix": _prefix(kvq, lens=None)}, 1),
                       ({"prefix": _prefix(kvq, groups=0)}, 1), ({"prefix": _prefix(kvq, groups=5)}, 1),
                       ({"prefix": _prefix(kvq, splits=-1)}, 1), ({"prefix": _prefix(kvq, splits=65)}, 1),
                       ({"prefix": _prefix(kvq, splits=40), "total": 160}, 1)):
        assert _plan(kvq, **over) == code, over


def _attend(kvq, **over):
    st = _struct(kvq)
    st.k_codes = st.v_codes = st.k_scales = st.v_scales = P
    a = dict(cache=st, q=P, batch=4, q_len=1, hq=24, scale=0.1, bt=P, width=20, sl=P, prefix=_prefix(kvq), plan=P,
             total=160, ctas=152, ws=P, ws_bytes=1 << 30, out=P, od=0, lse=None, flags=0)
    a.update(over)
    return kvq.lib().kvq_paged_prefix_attention(
        ctypes.byref(a["cache"]), a["q"], a["batch"], a["q_len"], a["hq"], a["scale"], a["bt"], a["width"], a["sl"],
        None if a["prefix"] is None else ctypes.byref(a["prefix"]), a["plan"], a["total"], a["ctas"], a["ws"],
        a["ws_bytes"], a["out"], a["od"], a["lse"], a["flags"], None)


def test_prefix_attention_refusals(kvq):
    g32 = _struct(kvq, "int8_g32")
    g32.k_codes = g32.v_codes = g32.k_scales = g32.v_scales = P
    for over, code in (({"q": None}, 1), ({"bt": None}, 1), ({"sl": None}, 1), ({"plan": None}, 1), ({"ws": None}, 1),
                       ({"out": None}, 1), ({"prefix": None}, 1), ({"batch": 0}, 1), ({"q_len": 0}, 1), ({"width": 0}, 1),
                       ({"hq": 0}, 1), ({"hq": 23}, 1), ({"hq": 36}, 2), ({"cache": g32}, 2), ({"od": 2}, 1),
                       ({"scale": float("nan")}, 1), ({"q": P + 8}, 1), ({"out": P + 8}, 1), ({"plan": P + 8}, 1),
                       ({"ws": P + 16}, 1), ({"ws_bytes": 4096}, 3), ({"total": 11}, 1), ({"ctas": 0}, 1),
                       ({"ctas": 153}, 1), ({"prefix": _prefix(kvq, splits=-1)}, 1), ({"prefix": _prefix(kvq, groups=5)}, 1)):
        assert _attend(kvq, **over) == code, over
    for flag in (2, 4, 8, 1 << 30):  # skip-merge, early start, rotate and the stall test belong to other calls
        assert _attend(kvq, flags=flag) == 1


def test_step_tables_keep_their_tensors(kvq):
    import torch

    t = kvq.StepTables.__new__(kvq.StepTables)
    object.__setattr__(t, "buffers", ())
    with pytest.raises(AttributeError):
        t.seq_lens = torch.zeros(4)


def test_shared_prefix_wants_one_offset_more(kvq):
    import torch

    with pytest.raises((ValueError, TypeError)):
        kvq.SharedPrefix(torch.zeros(3, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), 2)


def test_every_export_declares_its_arguments(kvq):
    """Addresses go to the library as Python integers: an entry without declared argument types would get 32 bits."""
    for name in kvq._binding.EXPORTS:
        assert getattr(kvq.lib(), name).argtypes is not None, name


def test_a_plan_with_shared_pages_is_for_prefix_decode(kvq):
    """decode and verify would leave the shared pages out: refused before anything is launched."""
    from types import SimpleNamespace as NS

    import torch

    from quantized_paged_kv_gb300 import cache as C

    q = torch.zeros(2, 1, 8, 128, dtype=torch.bfloat16)
    plan = NS(prefix=NS(splits=2), q_len=1)
    for call in (C.decode, C.verify):
        with pytest.raises(ValueError, match="prefix_decode"):
            call(None, plan, q, None, None, None, 1.0)
    for ok in (NS(), NS(prefix=None), NS(prefix=NS(splits=0))):
        C._own_pages_only(ok)


class _Fake:
    """What the binding asks of a tensor, on any device."""

    def __init__(self, dtype, shape, dev):  # dev -1: pinned host memory
        self.dtype, self.shape, self.dev, self.is_cuda = dtype, shape, dev, dev >= 0
        self.device = f"cuda:{dev}"

    def is_pinned(self):
        return self.dev < 0

    def dim(self):
        return len(self.shape)

    def get_device(self):
        return self.dev

    def is_contiguous(self):
        return True

    def numel(self):
        n = 1
        for x in self.shape:
            n *= x
        return n

    def data_ptr(self):
        return P


def test_arrays_on_another_device_are_refused(kvq, monkeypatch):
    """Before any launch: the cache, the group arrays and every tensor of a prefix call, the group arrays of a plan."""
    import torch

    B = kvq._binding
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    f = lambda dtype, *shape, dev=0: _Fake(dtype, shape, dev)
    i32, bf16, u8, f32 = torch.int32, torch.bfloat16, torch.uint8, torch.float32

    def attend(cache_dev=0, prefix_dev=0, **over):
        cache, prefix = _struct(kvq), _prefix(kvq)
        cache.device, prefix.device = cache_dev, prefix_dev
        a = dict(q=f(bf16, 4, 24, 256), bt=f(i32, 4, 20), sl=f(i32, 4), plan=f(i32, 10 ** 6), ws=f(u8, 1 << 30),
                 out=f(f32, 4, 24, 256), lse=f(f32, 4, 24))
        a.update(over)
        B.kvq_paged_prefix_attention(cache, a["q"], 0.1, a["bt"], a["sl"], prefix, a["plan"], 160, 152, a["ws"], a["out"],
                                     a["lse"], stream=type("S", (), {"cuda_stream": 0}))

    def plan(prefix_dev, sl=f(i32, 4)):
        prefix = _prefix(kvq)
        prefix.device = prefix_dev
        B.kvq_plan_splits_device(_struct(kvq), sl, 1, 20, prefix, 160, 152, f(i32, 10 ** 6), f(u8, 256),
                                 stream=type("S", (), {"cuda_stream": 0}))

    for over in ({"cache_dev": 1}, {"cache_dev": -1}, {"prefix_dev": 1}, {"q": f(bf16, 4, 24, 256, dev=1)},
                 {"bt": f(i32, 4, 20, dev=1)}, {"sl": f(i32, 4, dev=1)}, {"plan": f(i32, 10 ** 6, dev=1)},
                 {"ws": f(u8, 1 << 30, dev=1)}, {"out": f(f32, 4, 24, 256, dev=1)}, {"lse": f(f32, 4, 24, dev=1)}):
        with pytest.raises(ValueError, match="current device"):
            attend(**over)
    with pytest.raises(ValueError, match="current device"):
        plan(1)
    with pytest.raises(ValueError, match="current device"):
        plan(0, f(i32, 4, dev=1))


def test_a_prefix_knows_its_device(kvq, monkeypatch):
    import torch

    f = lambda dev, n: _Fake(torch.int32, (n,), dev)
    assert kvq.SharedPrefix(f(1, 3), f(1, 2), 2).struct.device == 1
    with pytest.raises(ValueError, match="different devices"):
        kvq.SharedPrefix(f(0, 3), f(1, 2), 2)
    assert kvq.KVCache("int8", 4, 1, 128, device="meta").struct.device == -1


def test_a_plan_is_for_its_own_prefix(kvq, monkeypatch):
    """prefix_decode takes the prefix that the plan was made with, or one over the same tensors: another one with the
    same number of splits would be read with offsets that the plan does not have."""
    from types import SimpleNamespace as NS

    import torch

    from quantized_paged_kv_gb300 import cache as C

    calls = []
    monkeypatch.setattr(kvq._binding, "kvq_paged_prefix_attention", lambda *a: calls.append(a))

    def prefix(offs, lens, splits=2):
        a, b = _Fake(torch.int32, (3,), 0), _Fake(torch.int32, (2,), 0)
        a.data_ptr, b.data_ptr = lambda: offs, lambda: lens
        return kvq.SharedPrefix(a, b, splits)

    q, bt = torch.zeros(4, 8, 128), torch.zeros(4, 20)
    made = prefix(P, P + 64)
    plan = NS(prefix=made, q_len=1, num_seqs=4, max_pages=20, plan=None, total_splits=0, num_ctas=0, workspace=None)
    call = lambda p: C.prefix_decode(NS(struct=None), plan, p, q, bt, None, None, 1.0)
    for ok in (made, prefix(P, P + 64)):
        call(ok)
    assert len(calls) == 2
    for other in (prefix(P + 256, P + 64), prefix(P, P + 128), prefix(P, P + 64, 3), prefix(P, P + 64, 0)):
        with pytest.raises(ValueError, match="without this prefix"):
            call(other)
    plan.prefix = prefix(P, P + 64, 0)  # nothing shared: the groups are not read
    call(prefix(P + 256, P + 512, 0))
    assert len(calls) == 3


def test_workspaces_and_plans_are_device_memory(kvq, monkeypatch):
    """Pinned host memory serves q, tables and lengths; what the kernels count and exchange partials in is the device's."""
    import torch

    B = kvq._binding
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    f = lambda dtype, *shape, dev=0: _Fake(dtype, shape, dev)
    i32, bf16, u8, f32 = torch.int32, torch.bfloat16, torch.uint8, torch.float32
    stream = type("S", (), {"cuda_stream": 0})
    with pytest.raises(ValueError, match="workspace must be device memory"):
        B.kvq_paged_prefix_attention(_struct(kvq), f(bf16, 4, 24, 256), 0.1, f(i32, 4, 20), f(i32, 4), _prefix(kvq),
                                     f(i32, 10 ** 6), 160, 152, f(u8, 1 << 30, dev=-1), f(f32, 4, 24, 256), stream=stream)
    for plan, status, name in ((f(i32, 10 ** 6, dev=-1), f(u8, 256), "plan"), (f(i32, 10 ** 6), f(u8, 256, dev=-1), "dev_status"),
                               (f(i32, 10 ** 6), torch.zeros(256, dtype=u8), "dev_status")):
        with pytest.raises(ValueError, match=name + " must be device memory"):
            B.kvq_plan_splits_device(_struct(kvq), f(i32, 4), 1, 20, None, 160, 152, plan, status, stream=stream)
    with pytest.raises(ValueError, match="workspace must be device memory"):
        B.tables_buffers(f(i32, 4, 10), f(torch.int64, 64), f(i32, 4), f(i32, 5), f(i32, 5), f(i32, 1), f(u8, 256, dev=-1))
    assert B.tables_buffers(f(i32, 4, 10), f(torch.int64, 64), f(i32, 4), f(i32, 5), f(i32, 5), f(i32, 1), f(u8, 256))[0] == 4


def test_nothing_shared_needs_no_groups(kvq):
    """splits = 0: NULL arrays and any group count pass the checks of both calls, up to those of the buffers' sizes
    (3), which come after."""
    for p in (_prefix(kvq, None, None, 0, 0), _prefix(kvq, None, None, 10 ** 9, 0), _prefix(kvq, P, P, -3, 0)):
        assert _plan(kvq, prefix=p, total=152, cap=100) == 3
        assert _attend(kvq, prefix=p, total=152, ws_bytes=4096) == 3
    assert _plan(kvq, prefix=_prefix(kvq, None, None, 0, -1)) == 1


def test_default_key_ranges_stay_short_enough_for_fp32(kvq):
    """The accumulator's truncation grows with a range's tokens: the default takes at most 4,096, as far as 64 ranges
    reach."""
    f = kvq.kvq_prefix_splits
    for fmt, hkv, hq, d in (("int8", 4, 24, 256), ("int8", 8, 32, 128), ("nvfp4", 2, 16, 256), ("bf16", 4, 28, 128)):
        s = _struct(kvq, fmt, hkv=hkv, d=d)
        for B, q in ((16, 1), (48, 1), (64, 6), (200, 4)):
            for n in (4096, 5000, 8192, 20000, 77777, 131072, 262144):
                S = f(s, B, q, hq, 1, n, 152)
                assert S == 0 or -(-n // 16) <= 256 * S, (fmt, B, q, n, S)
            assert f(s, B, q, hq, 1, 300000, 152) == 64


def test_a_device_plan_is_for_its_own_batch(kvq, monkeypatch):
    """decode and verify on a DevicePlan of another batch or query length: refused (on the GPU the plan's own check may
    take an offset for its CTA count)."""
    import torch

    from quantized_paged_kv_gb300 import cache as C

    calls = []
    for name in ("kvq_paged_decode_attention", "kvq_paged_verify_attention"):
        monkeypatch.setattr(kvq._binding, name, lambda *a: calls.append(a))

    class Plan:
        prefix, plan, total_splits, num_ctas, workspace = None, None, 0, 0, None

        def __init__(self, q_len, num_seqs):
            self.q_len, self.num_seqs = q_len, num_seqs

    cache = type("Cache", (), {"struct": None})
    one, three = torch.zeros(4, 8, 128), torch.zeros(4, 3, 8, 128)
    C.decode(cache, Plan(1, 4), one, None, None, None, 1.0)
    C.verify(cache, Plan(3, 4), three, None, None, None, 1.0)
    assert len(calls) == 2
    for plan in (Plan(1, 5), Plan(3, 4)):
        with pytest.raises(ValueError):
            C.decode(cache, plan, one, None, None, None, 1.0)
    for plan in (Plan(3, 5), Plan(1, 4)):
        with pytest.raises(ValueError):
            C.verify(cache, plan, three, None, None, None, 1.0)
    assert len(calls) == 2
