"""Device pools, split plans and workspaces around the C ABI (torch supplies the
device memory and the stream; every step of the path runs in libkvq's kernels).
"""
from __future__ import annotations

import torch

from . import _binding as B


class KVCache:
    """A paged K/V pool in one format, laid out as include/kvq.h documents:
    codes [num_pages][Hkv][16][row_bytes] and scales [num_pages][Hkv][16][...]
    for K and for V.  ``fill`` (a byte value) pre-fills every array, e.g. 0xFF
    so that unwritten slots hold NaN scales."""

    def __init__(self, fmt, num_pages, num_kv_heads, head_dim, page_size=16, device="cuda",
                 k_global_scale=1.0, v_global_scale=1.0, fill=None):
        self.fmt = fmt
        self.num_pages, self.num_kv_heads, self.head_dim, self.page_size = num_pages, num_kv_heads, head_dim, page_size
        cb, sb = B.kvq_cache_array_bytes(fmt, num_pages, page_size, num_kv_heads, head_dim)
        alloc = (lambda n: torch.empty(n, dtype=torch.uint8, device=device)) if fill is None else \
            (lambda n: torch.full((n,), fill, dtype=torch.uint8, device=device))
        self.k_codes, self.v_codes = alloc(cb), alloc(cb)
        self.k_scales, self.v_scales = (alloc(sb), alloc(sb)) if sb else (None, None)
        self.k_global_scale, self.v_global_scale = float(k_global_scale), float(v_global_scale)
        self.struct = B.KvqCacheStruct(
            self.k_codes.data_ptr(), self.v_codes.data_ptr(),
            self.k_scales.data_ptr() if sb else None, self.v_scales.data_ptr() if sb else None,
            num_pages, page_size, num_kv_heads, head_dim, B.FORMATS[fmt], self.k_global_scale, self.v_global_scale)
        self.struct.device = self.k_codes.get_device()

    @property
    def row_bytes(self):
        return {"bf16": 2 * self.head_dim, "int8": self.head_dim, "int8_g32": self.head_dim,
                "nvfp4": self.head_dim // 2}[self.fmt]

    def views(self):
        """(k_codes, v_codes, k_scales, v_scales) reshaped to [num_pages, Hkv, P, ...]."""
        shp = (self.num_pages, self.num_kv_heads, self.page_size)
        kc = self.k_codes.view(*shp, self.row_bytes)
        vc = self.v_codes.view(*shp, self.row_bytes)
        if self.k_scales is None:
            return kc, vc, None, None
        if self.fmt == "int8":
            return kc, vc, self.k_scales.view(torch.float32).view(*shp), self.v_scales.view(torch.float32).view(*shp)
        if self.fmt == "int8_g32":  # group-major: [num_pages, Hkv, D/32, P]
            gshp = (self.num_pages, self.num_kv_heads, self.head_dim // 32, self.page_size)
            return kc, vc, self.k_scales.view(torch.float32).view(*gshp), self.v_scales.view(torch.float32).view(*gshp)
        return kc, vc, self.k_scales.view(*shp, self.head_dim // 16), self.v_scales.view(*shp, self.head_dim // 16)

    def append(self, k_new, v_new, slot_mapping, dev_status=None, checked=False, rotate=False, stream=None):
        flags = (B.KVQ_CHECKED if checked else 0) | (B.KVQ_ROTATE if rotate else 0)
        B.kvq_quant_append(self.struct, k_new, v_new, slot_mapping, dev_status, flags, stream)


class DecodePlan:
    """Host split plan for one batch composition, copied to the device, plus the
    workspace it needs (status word zeroed once).  q_len > 1: the plan of a
    verify call over q_len query tokens a sequence."""

    def __init__(self, cache, seq_lens, num_q_heads, split_override=0, target_ctas=0, device="cuda", q_len=1):
        lens = [int(x) for x in seq_lens]
        if q_len == 1:
            plan, self.total_splits, self.num_ctas = B.kvq_plan_splits(cache.struct, lens, split_override, target_ctas)
        else:
            plan, self.total_splits, self.num_ctas = B.kvq_plan_verify_splits(cache.struct, lens, q_len,
                                                                              split_override, target_ctas)
        self.plan_host = plan
        self.plan = plan.to(device)
        self.q_len = q_len
        self.batch = len(seq_lens) * q_len
        self.num_q_heads = num_q_heads
        self.head_dim = cache.head_dim
        if q_len == 1:
            ws = B.kvq_decode_workspace_bytes(self.total_splits, num_q_heads, cache.head_dim)
        else:  # room for the tensor-core route of a one-sequence verify call as well
            ws = B.kvq_verify_workspace_bytes(cache.struct, len(seq_lens), q_len, num_q_heads, self.total_splits)
        self.workspace = torch.zeros(ws, dtype=torch.uint8, device=device)

    def partials(self):
        """(o_part pointer, lse_part pointer) inside the workspace."""
        return B.kvq_workspace_partials(self.workspace, self.total_splits, self.num_q_heads, self.head_dim)


def _own_pages_only(plan, num_seqs=None):
    prefix = getattr(plan, "prefix", None)
    if prefix is not None and prefix.splits:
        raise ValueError("the plan leaves shared pages out: use prefix_decode")
    made_for = getattr(plan, "num_seqs", num_seqs)  # a DevicePlan's
    if num_seqs is not None and made_for != num_seqs:
        raise ValueError(f"the plan is for {made_for} sequences, q has {num_seqs}")


def decode(cache, plan, q, block_tables, seq_lens, out, sm_scale, lse_out=None, checked=False, skip_merge=False,
           early_start=False, stream=None):
    """early_start: the plan and block tables are not written by the kernel just before this call on the stream
    (e.g. they were uploaded once for all layers of a step), so the decode may read them early."""
    _own_pages_only(plan, q.shape[0])
    if getattr(plan, "num_seqs", 0) and plan.q_len != 1:
        raise ValueError(f"the plan is for q_len {plan.q_len}: use verify")
    flags = ((B.KVQ_CHECKED if checked else 0) | (B.KVQ_SKIP_MERGE if skip_merge else 0)
             | (B.KVQ_EARLY_START if early_start else 0))
    B.kvq_paged_decode_attention(cache.struct, q, sm_scale, block_tables, seq_lens, plan.plan, plan.total_splits,
                                 plan.num_ctas, plan.workspace, out, lse_out, flags, stream)


def verify(cache, plan, q, block_tables, seq_lens, out, sm_scale, lse_out=None, checked=False, skip_merge=False,
           early_start=False, stream=None):
    """Causal attention for q.shape[1] query tokens a sequence; plan: DecodePlan(..., q_len=q.shape[1])."""
    _own_pages_only(plan, q.shape[0])
    if plan.q_len != q.shape[1]:
        raise ValueError(f"the plan is for q_len {plan.q_len}, q has {q.shape[1]} query tokens")
    flags = ((B.KVQ_CHECKED if checked else 0) | (B.KVQ_SKIP_MERGE if skip_merge else 0)
             | (B.KVQ_EARLY_START if early_start else 0))
    B.kvq_paged_verify_attention(cache.struct, q, sm_scale, block_tables, seq_lens, plan.plan, plan.total_splits,
                                 plan.num_ctas, plan.workspace, out, lse_out, flags, stream)


def prefill(cache, q, block_table, seq_len, out, sm_scale, lse_out=None, splits=0, workspace=None, checked=False,
            stream=None):
    """Causal attention of a prompt chunk: q [T, Hq, D] holds the last T of the sequence's seq_len tokens (their
    K/V already appended); block_table [max_pages] int32.  splits 0 = kvq_prefill_splits' choice.  Returns the
    workspace used (reusable for the same T / splits)."""
    T, Hq, D = q.shape
    if splits == 0:
        splits = B.kvq_prefill_splits(cache.struct, T, Hq, int(seq_len))
    need = B.kvq_prefill_workspace_bytes(T, Hq, D, splits)
    if workspace is None or workspace.numel() < need:
        workspace = torch.zeros(need, dtype=torch.uint8, device=q.device)
    B.kvq_paged_prefill_attention(cache.struct, q, sm_scale, block_table, seq_len, splits, workspace, out, lse_out,
                                  B.KVQ_CHECKED if checked else 0, stream)
    return workspace


class StepTables:
    """The device state that kvq_build_tables keeps for a batch: block_tables (int32 [batch, max_pages], the
    caller's), and its other outputs.  slot_mapping holds num_slots entries (-1 behind the step's last token).  The
    tensors are checked once, here, and stay: fill them in place (assigning another is refused)."""

    def __init__(self, block_tables, num_slots):
        B_, dev = block_tables.shape[0], block_tables.device
        i32 = lambda n: torch.zeros(n, dtype=torch.int32, device=dev)
        self.block_tables = block_tables
        self.slot_mapping = torch.full((num_slots,), -1, dtype=torch.int64, device=dev)
        self.seq_lens, self.query_start, self.page_start = i32(B_), i32(B_ + 1), i32(B_ + 1)
        self.free_head = i32(1)
        self.workspace = torch.zeros(B.KVQ_TABLES_WORKSPACE_BYTES, dtype=torch.uint8, device=dev)
        self.buffers = B.tables_buffers(self.block_tables, self.slot_mapping, self.seq_lens, self.query_start,
                                        self.page_start, self.free_head, self.workspace)

    def __setattr__(self, name, value):
        if "buffers" in self.__dict__:
            raise AttributeError(f"{name}: a StepTables keeps its tensors")
        object.__setattr__(self, name, value)


def build_tables(cache, tables, ctx_lens, new_lens, free_pages, free_head=None, checked=False, stream=None):
    """One step's block tables, slot map and lengths (kvq_build_tables) into ``tables``.  ctx_lens may be
    tables.seq_lens; free_head defaults to tables.free_head, which the call advances."""
    B.kvq_build_tables(cache.struct, ctx_lens, new_lens, free_pages,
                       tables.free_head if free_head is None else free_head, tables.buffers,
                       B.KVQ_CHECKED if checked else 0, stream)


class SharedPrefix:
    """The groups of a batch whose sequences share a prefix: int32 device tensors group_offsets [groups + 1] (group
    g = sequences group_offsets[g] .. group_offsets[g + 1] - 1) and prefix_lens [groups] (tokens), kept by reference;
    splits: key ranges of a prefix (prefix_splits gives a default; 0: the sequences read the pages each for
    itself)."""

    def __init__(self, group_offsets, prefix_lens, splits):
        B._need(group_offsets, torch.int32, "group_offsets")
        B._need(prefix_lens, torch.int32, "prefix_lens")
        if group_offsets.numel() != prefix_lens.numel() + 1:
            raise ValueError("group_offsets must hold one value more than prefix_lens")
        devices = {t.get_device() for t in (group_offsets, prefix_lens)} - {-1}
        if len(devices) > 1:
            raise ValueError("group_offsets and prefix_lens lie on different devices")
        self.group_offsets, self.prefix_lens, self.splits = group_offsets, prefix_lens, int(splits)
        struct = B.KvqPrefixStruct(group_offsets.data_ptr(), prefix_lens.data_ptr(), prefix_lens.numel(), self.splits)
        struct.device = devices.pop() if devices else -1
        # what a plan depends on (nothing of the groups where no page is shared)
        self.key = ((group_offsets.data_ptr(), prefix_lens.data_ptr(), prefix_lens.numel(), self.splits) if self.splits
                    else None)
        self.struct = struct

    def __setattr__(self, name, value):
        if "struct" in self.__dict__:
            raise AttributeError(f"{name}: a SharedPrefix keeps its tensors and splits")
        object.__setattr__(self, name, value)


def prefix_splits(cache, batch, num_q_heads, prefix_len, q_len=1, num_groups=1, target_ctas=0):
    """Key ranges for SharedPrefix: prefix_len = the longest prefix, in tokens; 0 where sharing is not expected to
    pay."""
    return B.kvq_prefix_splits(cache.struct, batch, q_len, num_q_heads, num_groups, int(prefix_len), target_ctas)


class DevicePlan:
    """A split plan made on the GPU from device lengths: update(seq_lens) writes it, on the stream, with no host
    work that depends on a length.  Takes the place of a DecodePlan in decode and verify; with ``prefix`` (a
    SharedPrefix) it is the plan of prefix_decode, and unless target_ctas is given the planner may make fewer splits
    of short own parts (KVQ_ONE_WAVE)."""

    def __init__(self, cache, batch, num_q_heads, max_pages, q_len=1, prefix=None, target_ctas=0, device="cuda"):
        self.cache, self.prefix, self.q_len, self.max_pages = cache, prefix, q_len, int(max_pages)
        self.num_seqs, self.batch = batch, batch * q_len
        self.num_q_heads, self.head_dim = num_q_heads, cache.head_dim
        self.flags = B.KVQ_ONE_WAVE if prefix and prefix.splits and not target_ctas else 0
        self.total_splits, self.num_ctas, entries = B.kvq_plan_device_sizes(
            cache.struct, batch, q_len, self.max_pages, prefix.splits if prefix else 0, target_ctas)
        self.plan = torch.zeros(entries, dtype=torch.int32, device=device)
        if q_len == 1 or (prefix and prefix.splits):
            ws = B.kvq_decode_workspace_bytes(self.total_splits, num_q_heads, cache.head_dim)
        else:
            ws = B.kvq_verify_workspace_bytes(cache.struct, batch, q_len, num_q_heads, self.total_splits)
        self.workspace = torch.zeros(ws, dtype=torch.uint8, device=device)

    def update(self, seq_lens, checked=False, stream=None):
        if seq_lens.numel() != self.num_seqs:
            raise ValueError(f"the plan is for {self.num_seqs} sequences, got {seq_lens.numel()} lengths")
        B.kvq_plan_splits_device(self.cache.struct, seq_lens, self.q_len, self.max_pages,
                                 self.prefix.struct if self.prefix else None, self.total_splits, self.num_ctas,
                                 self.plan, self.workspace, self.flags | (B.KVQ_CHECKED if checked else 0), stream)

    def partials(self):
        """(o_part pointer, lse_part pointer) inside the workspace."""
        return B.kvq_workspace_partials(self.workspace, self.total_splits, self.num_q_heads, self.head_dim)


def prefix_decode(cache, plan, prefix, q, block_tables, seq_lens, out, sm_scale, lse_out=None, checked=False,
                  stream=None):
    """Attention of a batch whose sequences share prefixes: q [B, Hq, D], or [B, q_len, Hq, D] (causal, as verify);
    plan: DevicePlan(..., prefix=prefix), updated with these lengths; prefix: the plan's, or another one over the same
    tensors."""
    if plan.prefix is not prefix and (plan.prefix is None or plan.prefix.key != prefix.key):
        raise ValueError("the plan was made without this prefix")
    T = q.shape[1] if q.dim() == 4 else 1
    if plan.q_len != T or plan.num_seqs != q.shape[0]:
        raise ValueError(f"the plan is for {plan.num_seqs} sequences of {plan.q_len} query tokens, q has "
                         f"{q.shape[0]} of {T}")
    if plan.max_pages != block_tables.shape[1]:
        raise ValueError(f"the plan is for block tables of {plan.max_pages} pages, got {block_tables.shape[1]}")
    B.kvq_paged_prefix_attention(cache.struct, q, sm_scale, block_tables, seq_lens, prefix.struct, plan.plan,
                                 plan.total_splits, plan.num_ctas, plan.workspace, out, lse_out,
                                 B.KVQ_CHECKED if checked else 0, stream)
