"""ctypes binding of libkvq.so — argument marshalling only.

Every function here has the name of the C entry point it calls (include/kvq.h)
and does nothing but turn torch tensors into device pointers, torch streams into
cudaStream_t handles, and non-zero status codes into exceptions.  All of the work
runs in the library's sm_103a kernels; there is no fallback: if libkvq.so is
missing, the first call raises.
"""
from __future__ import annotations

import ctypes
import os
from ctypes import POINTER, c_float, c_int32, c_int64, c_size_t, c_uint32, c_void_p

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_lib", "libkvq.so")

KVQ_FMT_BF16, KVQ_FMT_INT8, KVQ_FMT_NVFP4, KVQ_FMT_INT8_G32 = 0, 1, 2, 3
KVQ_OUT_F32, KVQ_OUT_BF16 = 0, 1
KVQ_CHECKED, KVQ_SKIP_MERGE, KVQ_EARLY_START = 1, 2, 4
KVQ_ROTATE = 8  # append: rotate each new K/V row (bf16(R(x))) before quantizing it
KVQ_ONE_WAVE = 16  # device plan with shared prefixes: one wave of splits where two would be short
KVQ_TEST_STALL = 1 << 30  # failure-path test: no page copies, every device wait gives up after 2 ms
KVQ_DEV_BAD_PAGE, KVQ_DEV_BAD_SEQLEN, KVQ_DEV_BAD_PLAN = 1, 2, 4
KVQ_DEV_TIMEOUT, KVQ_DEV_BAD_SLOT, KVQ_DEV_NONFINITE, KVQ_DEV_NO_PAGE = 8, 16, 32, 64
KVQ_TABLES_WORKSPACE_BYTES = 256
KVQ_STATIC_SCRATCH_BYTES = 16 << 20
FORMATS = {"bf16": KVQ_FMT_BF16, "int8": KVQ_FMT_INT8, "nvfp4": KVQ_FMT_NVFP4, "int8_g32": KVQ_FMT_INT8_G32}

# every symbol include/kvq.h declares
EXPORTS = (
    "kvq_bytes_per_token", "kvq_cache_array_bytes", "kvq_quant_append", "kvq_plan_splits", "kvq_plan_verify_splits",
    "kvq_decode_workspace_bytes", "kvq_verify_workspace_bytes", "kvq_workspace_partials", "kvq_paged_decode_attention",
    "kvq_paged_decode_attention_static", "kvq_paged_verify_attention", "kvq_prefill_splits",
    "kvq_prefill_workspace_bytes", "kvq_paged_prefill_attention", "kvq_split_merge", "kvq_read_status",
    "kvq_last_error", "kvq_rotate_rows", "kvq_build_tables", "kvq_prefix_splits", "kvq_plan_device_sizes",
    "kvq_plan_splits_device", "kvq_paged_prefix_attention",
)


class KvqCacheStruct(ctypes.Structure):
    _fields_ = [
        ("k_codes", c_void_p), ("v_codes", c_void_p), ("k_scales", c_void_p), ("v_scales", c_void_p),
        ("num_pages", c_int32), ("page_size", c_int32), ("num_kv_heads", c_int32), ("head_dim", c_int32),
        ("format", c_int32), ("k_global_scale", c_float), ("v_global_scale", c_float),
    ]


class KvqPrefixStruct(ctypes.Structure):
    _fields_ = [("group_offsets", c_void_p), ("prefix_lens", c_void_p), ("num_groups", c_int32), ("splits", c_int32)]


class KvqError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__(f"[kvq status {code}] {msg}")
        self.code = code


_lib = None


def lib():
    """Load libkvq.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                           "or python -m quantized_paged_kv_gb300.build")
    L = ctypes.CDLL(LIB_PATH)
    P = c_void_p
    sig = {
        "kvq_bytes_per_token": (c_int64, [c_int32, c_int32, c_int32]),
        "kvq_cache_array_bytes": (c_int32, [c_int32, c_int32, c_int32, c_int32, c_int32, POINTER(c_int64), POINTER(c_int64)]),
        "kvq_quant_append": (c_int32, [POINTER(KvqCacheStruct), P, P, P, c_int64, P, c_uint32, P]),
        "kvq_plan_splits": (c_int32, [POINTER(KvqCacheStruct), POINTER(c_int32), c_int32, c_int32, c_int32,
                                      POINTER(c_int32), c_int64, POINTER(c_int32), POINTER(c_int32)]),
        "kvq_plan_verify_splits": (c_int32, [POINTER(KvqCacheStruct), POINTER(c_int32), c_int32, c_int32, c_int32,
                                             c_int32, POINTER(c_int32), c_int64, POINTER(c_int32), POINTER(c_int32)]),
        "kvq_decode_workspace_bytes": (c_size_t, [c_int32, c_int32, c_int32]),
        "kvq_verify_workspace_bytes": (c_size_t, [POINTER(KvqCacheStruct), c_int32, c_int32, c_int32, c_int32,
                                                  c_int32]),
        "kvq_workspace_partials": (c_int32, [P, c_int32, c_int32, c_int32, POINTER(c_void_p), POINTER(c_void_p)]),
        "kvq_paged_decode_attention": (c_int32, [POINTER(KvqCacheStruct), P, c_int32, c_int32, c_float, P, c_int32,
                                                 P, P, c_int32, c_int32, P, c_size_t, P, c_int32, P, c_uint32, P]),
        "kvq_paged_decode_attention_static": (c_int32, [POINTER(KvqCacheStruct), P, c_int32, c_int32, c_float, P,
                                                        c_int32, P, P, c_int32, c_int32, P, c_int32, P, c_uint32, P]),
        "kvq_paged_verify_attention": (c_int32, [POINTER(KvqCacheStruct), P, c_int32, c_int32, c_int32, c_float, P,
                                                 c_int32, P, P, c_int32, c_int32, P, c_size_t, P, c_int32, P,
                                                 c_uint32, P]),
        "kvq_prefill_splits": (c_int32, [POINTER(KvqCacheStruct), c_int32, c_int32, c_int32, c_int32]),
        "kvq_prefill_workspace_bytes": (c_size_t, [c_int32, c_int32, c_int32, c_int32]),
        "kvq_paged_prefill_attention": (c_int32, [POINTER(KvqCacheStruct), P, c_int32, c_int32, c_float, P, c_int32,
                                                  c_int32, c_int32, P, c_size_t, P, c_int32, P, c_uint32, P]),
        "kvq_split_merge": (c_int32, [P, P, P, c_int32, c_int32, c_int32, P, c_int32, P, P]),
        "kvq_rotate_rows": (c_int32, [P, c_int32, P, c_int32, c_int64, c_int32, c_int32, P]),
        "kvq_build_tables": (c_int32, [POINTER(KvqCacheStruct), P, P, c_int32, P, c_int32, P, P, c_int32, P, c_int64, P,
                                       P, P, P, P, c_uint32, P]),
        "kvq_prefix_splits": (c_int32, [POINTER(KvqCacheStruct), c_int32, c_int32, c_int32, c_int32, c_int32,
                                        c_int32]),
        "kvq_plan_device_sizes": (c_int32, [POINTER(KvqCacheStruct), c_int32, c_int32, c_int32, c_int32, c_int32,
                                            POINTER(c_int32), POINTER(c_int32), POINTER(c_int64)]),
        "kvq_plan_splits_device": (c_int32, [POINTER(KvqCacheStruct), P, c_int32, c_int32, c_int32,
                                             POINTER(KvqPrefixStruct), c_int32, c_int32, P, c_int64, P, c_uint32, P]),
        "kvq_paged_prefix_attention": (c_int32, [POINTER(KvqCacheStruct), P, c_int32, c_int32, c_int32, c_float, P,
                                                 c_int32, P, POINTER(KvqPrefixStruct), P, c_int32, c_int32, P, c_size_t,
                                                 P, c_int32, P, c_uint32, P]),
        "kvq_read_status": (c_int32, [P, P, POINTER(c_int32)]),
        "kvq_last_error": (ctypes.c_char_p, []),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype, f.argtypes = res, args
    _lib = L
    return L


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is None:  # the current stream's handle, without building a Stream object for it
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream


def _check(rc, name):
    if rc != 0:
        raise KvqError(rc, f"{name}: {lib().kvq_last_error().decode()}")


def _shapes(q, out, lse_out, block_tables, seq_lens, cache_struct):
    """The buffers a device call writes or indexes, against q's shape (q is [B, ..., Hq, D]):
    out holds q's element count, lse_out one value a query row, block_tables and
    seq_lens a row per sequence."""
    if out.numel() != q.numel():
        raise ValueError(f"out must hold {q.numel()} values (q's shape {tuple(q.shape)}), got {tuple(out.shape)}")
    if lse_out is not None and lse_out.numel() != q.numel() // q.shape[-1]:
        raise ValueError(f"lse_out must hold {q.numel() // q.shape[-1]} values, got {tuple(lse_out.shape)}")
    if q.shape[-1] != cache_struct.head_dim:
        raise ValueError(f"q's head_dim {q.shape[-1]} != the cache's {cache_struct.head_dim}")
    if block_tables is not None and (block_tables.dim() != 2 or block_tables.shape[0] < q.shape[0]):
        raise ValueError(f"block_tables must be [>= {q.shape[0]}, max_pages]")
    if seq_lens is not None and seq_lens.numel() < q.shape[0]:
        raise ValueError(f"seq_lens must hold {q.shape[0]} lengths")


def _need(t, dtype, name, device=True):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device and not (t.is_cuda or t.is_pinned()):
        raise ValueError(f"{name} must be a CUDA tensor or pinned host memory")


def _device(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be device memory")


def _here(*tensors):
    """The tensors of one call lie on the current device (pinned host memory aside)."""
    cur = torch._C._cuda_getDevice()
    for t in tensors:
        if t is not None and t.is_cuda and t.get_device() != cur:
            raise ValueError(f"a tensor on {t.device}, the current device is cuda:{cur}")


def _struct_here(struct, name, cur, pinned=-1):
    """The arrays behind a struct lie on device cur or, where that is allowed, in pinned host memory (KVCache and
    SharedPrefix note the device, -1 for the host)."""
    dev = getattr(struct, "device", cur)
    if dev != cur and dev != pinned:
        raise ValueError(f"{name} lies on {'the host' if dev < 0 else f'cuda:{dev}'}, the current device is cuda:{cur}")


def _on(t, dtype, name, cur):
    """t is contiguous, of dtype, on device cur or in pinned host memory."""
    if t.dtype is not dtype or not t.is_contiguous() or t.get_device() != cur:
        _need(t, dtype, name)
        _here(t)


def _int32(t, n, name, cur):
    """t's address: int32, contiguous, n values (None: any number), on device cur or pinned host memory."""
    if t.dtype is not torch.int32 or not t.is_contiguous() or t.get_device() != cur:
        _need(t, torch.int32, name)
        _here(t)
    if n is not None and t.numel() != n:
        raise ValueError(f"{name} must hold {n} values, got {t.numel()}")
    return t.data_ptr()


# ----------------------------------------------------------------- host helpers
def kvq_bytes_per_token(fmt, num_kv_heads, head_dim):
    return int(lib().kvq_bytes_per_token(FORMATS.get(fmt, fmt), num_kv_heads, head_dim))


def kvq_cache_array_bytes(fmt, num_pages, page_size, num_kv_heads, head_dim):
    cb, sb = c_int64(), c_int64()
    _check(lib().kvq_cache_array_bytes(FORMATS.get(fmt, fmt), num_pages, page_size, num_kv_heads, head_dim,
                                       ctypes.byref(cb), ctypes.byref(sb)), "kvq_cache_array_bytes")
    return cb.value, sb.value


def kvq_decode_workspace_bytes(total_splits, num_q_heads, head_dim):
    return int(lib().kvq_decode_workspace_bytes(total_splits, num_q_heads, head_dim))


def kvq_verify_workspace_bytes(cache_struct, batch, q_len, num_q_heads, total_splits, target_ctas=0):
    """Workspace bytes of a verify call, the tensor-core route of a one-sequence call included."""
    n = int(lib().kvq_verify_workspace_bytes(ctypes.byref(cache_struct), batch, q_len, num_q_heads, total_splits,
                                             target_ctas))
    if n == 0:
        raise KvqError(1, f"kvq_verify_workspace_bytes: {lib().kvq_last_error().decode()}")
    return n


def _plan(call, name, cache_struct, seq_lens, lead, split_override, target_ctas, virtual_batch):
    """A size query, then the plan itself; ``lead`` = the arguments between
    seq_lens and split_override (the batch, and q_len for a verify plan)."""
    sl = torch.as_tensor(list(seq_lens), dtype=torch.int32)
    total, nctas = c_int32(), c_int32()
    slp = sl.numpy().ctypes.data_as(POINTER(c_int32))
    rc = call(ctypes.byref(cache_struct), slp, *lead, split_override, target_ctas, None, 0, ctypes.byref(total),
              ctypes.byref(nctas))
    if rc not in (0, 3):  # 3 = KVQ_ERR_WORKSPACE (size query)
        _check(rc, name)
    # head groups per split <= num_kv_heads, so this bounds the plan length
    plan = torch.zeros(virtual_batch + 9 + nctas.value + 4 * total.value * cache_struct.num_kv_heads,
                       dtype=torch.int32)
    _check(call(ctypes.byref(cache_struct), slp, *lead, split_override, target_ctas,
                plan.numpy().ctypes.data_as(POINTER(c_int32)), plan.numel(), ctypes.byref(total),
                ctypes.byref(nctas)), name)
    return plan, total.value, nctas.value


def kvq_plan_splits(cache_struct, seq_lens, split_override=0, target_ctas=0):
    """seq_lens: host int sequence.  Returns (plan int32 CPU tensor, total_splits, num_ctas)."""
    B = len(seq_lens)
    return _plan(lib().kvq_plan_splits, "kvq_plan_splits", cache_struct, seq_lens, (B,), split_override,
                 target_ctas, B)


def kvq_plan_verify_splits(cache_struct, seq_lens, q_len, split_override=0, target_ctas=0):
    """The plan of a verify call over q_len query tokens a sequence (the causal
    visible lengths are computed by the library)."""
    B = len(seq_lens)
    return _plan(lib().kvq_plan_verify_splits, "kvq_plan_verify_splits", cache_struct, seq_lens, (B, q_len),
                 split_override, target_ctas, B * q_len)


def kvq_workspace_partials(workspace, total_splits, num_q_heads, head_dim):
    o, l = c_void_p(), c_void_p()
    _check(lib().kvq_workspace_partials(_ptr(workspace), total_splits, num_q_heads, head_dim, ctypes.byref(o),
                                        ctypes.byref(l)), "kvq_workspace_partials")
    return o.value, l.value


def kvq_read_status(dev_status, stream=None):
    """Returns (status code, bits) without raising."""
    bits = c_int32()
    rc = lib().kvq_read_status(_ptr(dev_status), _stream(stream), ctypes.byref(bits))
    return rc, bits.value


def kvq_last_error():
    return lib().kvq_last_error().decode()


# ----------------------------------------------------------------- device calls
def kvq_quant_append(cache_struct, k_new, v_new, slot_mapping, dev_status=None, flags=0, stream=None):
    _need(k_new, torch.bfloat16, "k_new")
    _need(v_new, torch.bfloat16, "v_new")
    _need(slot_mapping, torch.int64, "slot_mapping")
    n = slot_mapping.numel()
    if k_new.shape != v_new.shape or k_new.shape[0] != n:
        raise ValueError("k_new / v_new must be [n_tokens, Hkv, D] and match slot_mapping")
    _check(lib().kvq_quant_append(ctypes.byref(cache_struct), _ptr(k_new), _ptr(v_new), _ptr(slot_mapping), n,
                                  _ptr(dev_status), flags, _stream(stream)), "kvq_quant_append")


def kvq_paged_decode_attention(cache_struct, q, sm_scale, block_tables, seq_lens, plan, total_splits, num_ctas,
                               workspace, out, lse_out=None, flags=0, stream=None):
    _need(q, torch.bfloat16, "q")
    _need(block_tables, torch.int32, "block_tables")
    _need(seq_lens, torch.int32, "seq_lens")
    _need(plan, torch.int32, "plan")
    _need(workspace, torch.uint8, "workspace")
    if out.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("out must be float32 or bfloat16")
    _need(out, out.dtype, "out")
    if lse_out is not None:
        _need(lse_out, torch.float32, "lse_out")
    _shapes(q, out, lse_out, block_tables, seq_lens, cache_struct)
    B, Hq, _ = q.shape
    od = KVQ_OUT_BF16 if out.dtype == torch.bfloat16 else KVQ_OUT_F32
    _check(lib().kvq_paged_decode_attention(
        ctypes.byref(cache_struct), _ptr(q), B, Hq, float(sm_scale), _ptr(block_tables), block_tables.shape[1],
        _ptr(seq_lens), _ptr(plan), total_splits, num_ctas, _ptr(workspace), workspace.numel(), _ptr(out), od,
        _ptr(lse_out),
        flags, _stream(stream)), "kvq_paged_decode_attention")


def kvq_paged_decode_attention_static(cache_struct, q, sm_scale, block_tables, seq_lens, plan, total_splits,
                                      num_ctas, out, lse_out=None, flags=0, stream=None):
    """kvq_paged_decode_attention with the library's static scratch region in place of a workspace."""
    _need(q, torch.bfloat16, "q")
    _need(block_tables, torch.int32, "block_tables")
    _need(seq_lens, torch.int32, "seq_lens")
    _need(plan, torch.int32, "plan")
    if out.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("out must be float32 or bfloat16")
    _need(out, out.dtype, "out")
    if lse_out is not None:
        _need(lse_out, torch.float32, "lse_out")
    _shapes(q, out, lse_out, block_tables, seq_lens, cache_struct)
    B, Hq, _ = q.shape
    od = KVQ_OUT_BF16 if out.dtype == torch.bfloat16 else KVQ_OUT_F32
    _check(lib().kvq_paged_decode_attention_static(
        ctypes.byref(cache_struct), _ptr(q), B, Hq, float(sm_scale), _ptr(block_tables), block_tables.shape[1],
        _ptr(seq_lens), _ptr(plan), total_splits, num_ctas, _ptr(out), od, _ptr(lse_out), flags, _stream(stream)),
        "kvq_paged_decode_attention_static")


def kvq_paged_verify_attention(cache_struct, q, sm_scale, block_tables, seq_lens, plan, total_splits, num_ctas,
                               workspace, out, lse_out=None, flags=0, stream=None):
    """q: bf16 [B, q_len, Hq, D]; out: [B, q_len, Hq, D]; lse_out: [B, q_len, Hq]."""
    _need(q, torch.bfloat16, "q")
    _need(block_tables, torch.int32, "block_tables")
    _need(seq_lens, torch.int32, "seq_lens")
    _need(plan, torch.int32, "plan")
    _need(workspace, torch.uint8, "workspace")
    if out.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("out must be float32 or bfloat16")
    _need(out, out.dtype, "out")
    if lse_out is not None:
        _need(lse_out, torch.float32, "lse_out")
    _shapes(q, out, lse_out, block_tables, seq_lens, cache_struct)
    B, T, Hq, _ = q.shape
    od = KVQ_OUT_BF16 if out.dtype == torch.bfloat16 else KVQ_OUT_F32
    _check(lib().kvq_paged_verify_attention(
        ctypes.byref(cache_struct), _ptr(q), B, T, Hq, float(sm_scale), _ptr(block_tables), block_tables.shape[1],
        _ptr(seq_lens), _ptr(plan), total_splits, num_ctas, _ptr(workspace), workspace.numel(), _ptr(out), od,
        _ptr(lse_out), flags, _stream(stream)), "kvq_paged_verify_attention")


def kvq_prefill_splits(cache_struct, q_len, num_q_heads, seq_len, target_ctas=0):
    n = int(lib().kvq_prefill_splits(ctypes.byref(cache_struct), q_len, num_q_heads, seq_len, target_ctas))
    if n < 1:
        _check(-n, "kvq_prefill_splits")
    return n


def kvq_prefill_workspace_bytes(q_len, num_q_heads, head_dim, splits):
    return int(lib().kvq_prefill_workspace_bytes(q_len, num_q_heads, head_dim, splits))


def kvq_paged_prefill_attention(cache_struct, q, sm_scale, block_table, seq_len, splits, workspace, out,
                                lse_out=None, flags=0, stream=None):
    """q: bf16 [T, Hq, D] (the last T tokens of the sequence); block_table: int32 [max_pages]."""
    _need(q, torch.bfloat16, "q")
    _need(block_table, torch.int32, "block_table")
    _need(workspace, torch.uint8, "workspace")
    if out.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("out must be float32 or bfloat16")
    _need(out, out.dtype, "out")
    if lse_out is not None:
        _need(lse_out, torch.float32, "lse_out")
    _shapes(q, out, lse_out, None, None, cache_struct)
    T, Hq, _ = q.shape
    od = KVQ_OUT_BF16 if out.dtype == torch.bfloat16 else KVQ_OUT_F32
    _check(lib().kvq_paged_prefill_attention(
        ctypes.byref(cache_struct), _ptr(q), T, Hq, float(sm_scale), _ptr(block_table), block_table.numel(),
        int(seq_len), splits, _ptr(workspace), workspace.numel(), _ptr(out), od, _ptr(lse_out), flags,
        _stream(stream)), "kvq_paged_prefill_attention")


def kvq_split_merge(o_part_ptr, lse_part_ptr, split_offsets, batch, num_q_heads, head_dim, out, lse_out=None,
                    stream=None):
    od = KVQ_OUT_BF16 if out.dtype == torch.bfloat16 else KVQ_OUT_F32
    _check(lib().kvq_split_merge(c_void_p(o_part_ptr), c_void_p(lse_part_ptr), _ptr(split_offsets), batch,
                                 num_q_heads, head_dim, _ptr(out), od, _ptr(lse_out), _stream(stream)),
           "kvq_split_merge")


def kvq_rotate_rows(x, out=None, inverse=False, stream=None):
    """out[..., :] = R(x[..., :]) (or R^-1) over the last axis (head_dim 128 / 256);
    x and out float32 or bfloat16, device or pinned host; out defaults to a new
    tensor of x's dtype on x's device (out may be x)."""
    if x.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("x must be float32 or bfloat16")
    if out is None:
        out = torch.empty_like(x)
    if out.dtype not in (torch.float32, torch.bfloat16) or out.shape != x.shape:
        raise TypeError("out must be float32 or bfloat16 with x's shape")
    if not x.is_contiguous() or not out.is_contiguous():
        raise ValueError("x and out must be contiguous")
    D = x.shape[-1]
    dt = lambda t: KVQ_OUT_BF16 if t.dtype == torch.bfloat16 else KVQ_OUT_F32
    _check(lib().kvq_rotate_rows(_ptr(x), dt(x), _ptr(out), dt(out), ctypes.c_int64(x.numel() // max(D, 1)), D,
                                 1 if inverse else 0, _stream(stream)), "kvq_rotate_rows")
    return out


def tables_buffers(block_tables, slot_mapping, seq_lens, query_start, page_start, free_head_out, workspace):
    """The checked addresses and sizes of the buffers that kvq_build_tables writes, for its ``buffers`` argument:
    int32 on the device but slot_mapping (int64) and workspace (uint8)."""
    if block_tables.dim() != 2:
        raise ValueError("block_tables must be [batch, max_pages]")
    n = block_tables.shape[0]
    dev = block_tables.get_device()
    _need(block_tables, torch.int32, "block_tables")
    _need(slot_mapping, torch.int64, "slot_mapping")
    _need(workspace, torch.uint8, "workspace")
    _device(workspace, "workspace")
    for t, m, name in ((seq_lens, n, "seq_lens"), (query_start, n + 1, "query_start"), (page_start, n + 1, "page_start"),
                       (free_head_out, 1, "free_head_out")):
        _int32(t, m, name, dev)
    if any(t.is_cuda and t.get_device() != dev for t in (slot_mapping, workspace)):
        raise ValueError("the buffers lie on different devices")
    if workspace.numel() < KVQ_TABLES_WORKSPACE_BYTES:
        raise ValueError(f"workspace must hold {KVQ_TABLES_WORKSPACE_BYTES} bytes")
    P = c_void_p
    return (n, dev, P(block_tables.data_ptr()), c_int32(block_tables.shape[1]), P(slot_mapping.data_ptr()),
            c_int64(slot_mapping.numel()), P(seq_lens.data_ptr()), P(query_start.data_ptr()), P(page_start.data_ptr()),
            P(free_head_out.data_ptr()), P(workspace.data_ptr()))


def kvq_build_tables(cache_struct, ctx_lens, new_lens, free_pages, free_head, buffers, flags=0, stream=None):
    """buffers: tables_buffers(...) of the outputs; the other tensors int32 on the device."""
    n, dev, bt, width, slots, num_slots, sl, qs, ps, head_out, ws = buffers
    cur = torch._C._cuda_getDevice()
    if dev != cur:
        raise ValueError(f"the buffers lie on cuda:{dev}, the current device is cuda:{cur}")
    _check(lib().kvq_build_tables(
        ctypes.byref(cache_struct), _int32(ctx_lens, n, "ctx_lens", cur), _int32(new_lens, n, "new_lens", cur), n,
        _int32(free_pages, None, "free_pages", cur), free_pages.numel(), _int32(free_head, 1, "free_head", cur), bt,
        width, slots, num_slots, sl, qs, ps, head_out, ws, flags, _stream(stream)), "kvq_build_tables")


def kvq_prefix_splits(cache_struct, batch, q_len, num_q_heads, num_groups, prefix_len, target_ctas=0):
    n = int(lib().kvq_prefix_splits(ctypes.byref(cache_struct), batch, q_len, num_q_heads, num_groups, prefix_len,
                                    target_ctas))
    if n < 0:
        _check(-n, "kvq_prefix_splits")
    return n


def kvq_plan_device_sizes(cache_struct, batch, q_len, max_pages, prefix_splits=0, target_ctas=0):
    """(total_splits, num_ctas, int32 entries of the plan)."""
    total, nctas, entries = c_int32(), c_int32(), c_int64()
    _check(lib().kvq_plan_device_sizes(ctypes.byref(cache_struct), batch, q_len, max_pages, prefix_splits, target_ctas,
                                       ctypes.byref(total), ctypes.byref(nctas), ctypes.byref(entries)),
           "kvq_plan_device_sizes")
    return total.value, nctas.value, entries.value


def kvq_plan_splits_device(cache_struct, seq_lens, q_len, max_pages, prefix_struct, total_splits, num_ctas, plan,
                           dev_status, flags=0, stream=None):
    """prefix_struct: a KvqPrefixStruct or None; plan: int32 on the device; dev_status: any device word."""
    cur = torch._C._cuda_getDevice()
    plan_ptr = _int32(plan, None, "plan", cur)
    _device(plan, "plan")
    _device(dev_status, "dev_status")
    _here(dev_status)
    if prefix_struct is not None:
        _struct_here(prefix_struct, "the prefix", cur)
    _check(lib().kvq_plan_splits_device(
        ctypes.byref(cache_struct), _int32(seq_lens, None, "seq_lens", cur), seq_lens.numel(), q_len, max_pages,
        None if prefix_struct is None else ctypes.byref(prefix_struct), total_splits, num_ctas, plan_ptr,
        plan.numel(), _ptr(dev_status), flags, _stream(stream)), "kvq_plan_splits_device")


def kvq_paged_prefix_attention(cache_struct, q, sm_scale, block_tables, seq_lens, prefix_struct, plan, total_splits,
                               num_ctas, workspace, out, lse_out=None, flags=0, stream=None):
    """q, out: [B, Hq, D], or [B, q_len, Hq, D]; lse_out: [B, Hq] / [B, q_len, Hq]."""
    cur = torch._C._cuda_getDevice()
    odt = out.dtype
    if odt is not torch.bfloat16:
        odt = torch.float32
    _struct_here(cache_struct, "the cache", cur, pinned=cur)
    _struct_here(prefix_struct, "the prefix", cur)
    _on(q, torch.bfloat16, "q", cur)
    _on(out, odt, "out", cur)
    _on(workspace, torch.uint8, "workspace", cur)
    _device(workspace, "workspace")
    if lse_out is not None:
        _on(lse_out, torch.float32, "lse_out", cur)
    bt, sl, pl = (_int32(block_tables, None, "block_tables", cur), _int32(seq_lens, None, "seq_lens", cur),
                  _int32(plan, None, "plan", cur))
    shape, n, width = q.shape, q.numel(), block_tables.shape
    if len(shape) == 4:
        B, T, Hq, D = shape
    elif len(shape) == 3:
        B, Hq, D = shape
        T = 1
    else:
        raise ValueError("q must be [B, Hq, D] or [B, q_len, Hq, D]")
    if (out.numel() != n or D != cache_struct.head_dim or len(width) != 2 or width[0] < B or seq_lens.numel() < B
            or (lse_out is not None and lse_out.numel() * D != n)):
        _shapes(q, out, lse_out, block_tables, seq_lens, cache_struct)
    od = KVQ_OUT_BF16 if odt is torch.bfloat16 else KVQ_OUT_F32
    _check(lib().kvq_paged_prefix_attention(
        ctypes.byref(cache_struct), q.data_ptr(), B, T, Hq, float(sm_scale), bt, width[1], sl,
        ctypes.byref(prefix_struct), pl, total_splits, num_ctas, workspace.data_ptr(), workspace.numel(),
        out.data_ptr(), od, _ptr(lse_out), flags, _stream(stream)), "kvq_paged_prefix_attention")
