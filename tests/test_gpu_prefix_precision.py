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
