"""How exact kvq_paged_prefix_attention's fp32 output is, and its bf16 output where V scales of one tile lie far apart.

Tolerance, fp32 output, as a 2-norm over the output.  The tensor cores' accumulator truncates: half a unit of 2^-23 in the
mean, always towards zero, at each of the products with 16 keys, of which there are two (hi and lo) a step, so n keys of a
range make n / 8 steps and an error of up to n / 8 x 2^-24 of the output.  P as two 11-bit terms leaves 2^-22 and as two
bf16 terms 2^-18 (one key's weight; both at most), fp32 logits, weights and sums a few 2^-23: 2^-20 for all of them, 2^-17
on a BF16 cache.  One term of P alone would leave 2^-12 (fp16) and 2^-9 (bf16)."""
import numpy as np
import pytest
import torch

from oracle import attention as oatt
from quantized_paged_kv_gb300 import workloads as W
from tests import harness as H
from tests.test_gpu_prefix import _Call, _one_group

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    H.ensure_built()


@pytest.mark.parametrize("fmt", ["int8", "nvfp4", "bf16"])
@pytest.mark.parametrize("name", ["tiny_int8", "serving_int8"])
@pytest.mark.parametrize("n,splits", [(512, 1), (4096, 1), (4096, 8)])
def test_fp32_output_by_tokens_of_a_range(fmt, name, n, splits):
    wl = _one_group(name, [n, n, n], n, 101)
    gs = H.global_scales(wl, fmt)
    c = _Call(wl, fmt, [0, 3], [n], splits=splits, gs=gs)
    c.launch(checked=True)
    heads = (0, wl.Hkv - 1)
    ref, ref_lse = oatt.paged_verify(fmt, H.oracle_pools(wl, fmt, gs, heads=heads), c.q, wl.block_tables, wl.seq_lens,
                                     wl.sm_scale, units=[(b, 0, h) for b in range(3) for h in heads])
    rows = ~np.isnan(ref_lse)
    d = c.out.cpu().numpy()[rows].astype(np.float64) - ref[rows]
    bound = n / splits / 8 * 2.0 ** -24 + (2.0 ** -17 if fmt == "bf16" else 2.0 ** -20)
    assert np.linalg.norm(d) <= bound * np.linalg.norm(ref[rows]), np.linalg.norm(d) / np.linalg.norm(ref[rows])
    # lse: logits and sums in fp32, of size up to 2^5
    assert np.abs(c.lse.cpu().numpy()[rows] - ref_lse[rows]).max() <= 2.0 ** -17


@pytest.mark.parametrize("ratio", [2.0 ** -10, 2.0 ** -14, 2.0 ** -18])
@pytest.mark.parametrize("out_dtype", ["f32", "bf16"])
def test_int8_v_of_two_sizes_in_every_tile(ratio, out_dtype):
    """V alternates between sizes 1 and `ratio` from token to token; one query of each row of heads weighs a small token
    most, one a large token.  Beside the relative terms (bf16: 2^-8 of the output, three fp16 roundings of 2^-11 a key;
    fp32: the accumulator's n / 8 x 2^-23 and 2^-20) a key's factor is off by fp16's smallest number, 2^-25 of a unit of
    at most twice the largest scale: w x 2^-23 max |V| for V's factor and product, and for the weight, whose sum is at
    least 1/2, 2^-23 max |V|, or all of the key where that is less."""
    n = 704
    wl = _one_group("tiny_int8", [n, n, n], n, 102)
    plain = wl.kv
    wl.kv = lambda b: (plain(b)[0], W.bf16_round(plain(b)[1] * np.where(np.arange(n) % 2, ratio, 1.0)[:, None, None]))
    q = wl.q_tokens(1)
    G = wl.Hq // wl.Hkv
    for b, token in ((0, 301), (1, 300)):
        q[b, 0] += np.repeat(plain(2)[0][token], G, 0).reshape(wl.Hq, wl.D)
    q = W.bf16_round(q)
    c = _Call(wl, "int8", [0, 3], [n], splits=1, out_dtype=out_dtype, q=q)
    c.launch(checked=True)
    out = c.out.float().cpu().numpy()[:, 0].astype(np.float64)
    pools = H.oracle_pools(wl, "int8")
    for b in range(3):
        slots = wl.slots(b)
        for h in range(wl.Hkv):
            k = oatt.cache_rows("int8", pools["k_codes"], pools["k_scales"], slots, h)
            v = oatt.cache_rows("int8", pools["v_codes"], pools["v_scales"], slots, h)
            z = np.asarray(q[b, 0, G * h:G * h + G], np.float64) @ k.T * wl.sm_scale
            w = np.exp(z - z.max(-1, keepdims=True))
            w /= w.sum(-1, keepdims=True)
            ref, size, vmax = w @ v, w @ np.abs(v), np.abs(v).max()
            rel = 2.0 ** -8 * np.abs(ref) + 3 * 2.0 ** -11 * size if out_dtype == "bf16" else \
                (n / 8 * 2.0 ** -23 + 2.0 ** -20) * size
            lost = np.stack([np.minimum(2.0 ** -23 * vmax, 2 * w[g][:, None] * np.abs(v)).sum(0) for g in range(G)])
            bound = rel + 2e-5 * size + 2.0 ** -23 * vmax + lost
            d = np.abs(out[b, G * h:G * h + G] - ref)
            assert np.all(d <= bound), (d / bound).max()


@pytest.mark.parametrize("T,splits,own", [(1, 2, 120), (1, 1, 0), (1, 0, 120), (6, 0, 120), (3, 2, 120)])
@pytest.mark.parametrize("name", ["tiny_int8", "serving_int8"])
def test_bf16_output_of_a_bf16_cache_is_the_rounded_result(T, splits, own, name):
    """Shared and own pages, nothing shared (T = 6: the tensor-core route of several query tokens): the output is within
    half a bf16 step of the result and what fp32 output is off by: n / 8 x 2^-23 (at most one unit a product) and 2^-17
    of sum w |v|.  One bf16 term of P would add up to 2^-9 (half a step of a number in [1, 2), relative to 1) a weight."""
    n = 704
    wl = _one_group(name, [n + own, n + own // 2, n], n, 105)
    c = _Call(wl, "bf16", [0, 3], [n], T=T, splits=splits, out_dtype="bf16")
    c.launch(checked=True)
    pools = H.oracle_pools(wl, "bf16")
    flat = dict(pools, v_codes=(pools["v_codes"].view(np.uint16) & 0x7FFF).view(np.uint8))
    verify = lambda p: oatt.paged_verify("bf16", p, c.q, wl.block_tables, wl.seq_lens, wl.sm_scale)[0]
    ref, size = verify(pools), verify(flat)
    step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(ref), 1e-30))) - 7)
    # a result just below a power of two may be rounded in the upper binade's steps
    bound = step / 2 * 2.0 ** (np.abs(ref) > 0.999 * 2 ** 8 * step) + ((n + own) / 8 * 2.0 ** -23 + 2.0 ** -17) * size
    d = np.abs(c.out.float().cpu().numpy() - ref)
    assert np.all(d <= bound), (d / bound).max()
