"""kvq_paged_prefix_attention where single values are unlike the rest: runs of V = 0, V near the ends of its range.

Tolerance, fp32 output: as in test_gpu_prefix_range.py, 2e-3 times the size of V.  bf16 output, INT8 cache, with w the
softmax weights: the output's rounding, 2^-8 |out| (half a step of bf16), plus three fp16 roundings of 2^-11 a key (of
its weight, of its V scale, of their product with the code), 3 x 2^-11 sum w |v|, plus fp16's smallest number: a factor
below 2^-14 is off by up to 2^-25 of its unit, which is at most twice the largest V scale.  With codes up to 127 and
max |V| = 127 x the largest scale that is 2^-24 max |V| for the V factor and its product, weighted (twice 2^-24 in all),
and 2^-24 max |V| a key for the weight, over a sum of weights of at least 1/2: n x 2^-23 max |V|.  2e-5 sum w |v| stands
for the logits' and the sums' fp32 arithmetic."""
import numpy as np
import pytest
import torch

from oracle import attention as oatt
from quantized_paged_kv_gb300 import workloads as W
from tests import harness as H
from tests.test_gpu_prefix import _Call, _one_group, _share
from tests.test_gpu_prefix_range import _scale_v

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    H.ensure_built()


def _check(c, size, pools=None):
    """c's outputs against the oracle's (over its own pools, or those given)."""
    wl = c.wl
    pools = H.oracle_pools(wl, c.fmt, c.gs) if pools is None else pools
    verify = lambda p: oatt.paged_verify(c.fmt, p, c.q, wl.block_tables, wl.seq_lens, wl.sm_scale)
    ref, ref_lse = verify(pools)
    out = c.out.float().cpu().numpy()
    assert np.all(np.isfinite(out))
    bound = 2e-3 * size
    if c.out_dtype == "bf16":
        assert c.fmt == "int8"
        flat = dict(pools, v_codes=np.abs(pools["v_codes"].view(np.int8).astype(np.int16)).astype(np.uint8),
                    v_scales=np.abs(pools["v_scales"]))
        weighted, _ = verify(flat)  # sum of w |v|
        vmax = 127 * np.nanmax(flat["v_scales"])
        n = int(wl.seq_lens.max())
        bound = 2.0 ** -8 * np.abs(ref) + (3 * 2.0 ** -11 + 2e-5) * weighted + (n + 1) * 2.0 ** -23 * vmax
    assert np.all(np.abs(out - ref) <= bound), (np.abs(out - ref) / bound).max()
    assert np.abs(c.lse.cpu().numpy() - ref_lse).max() < 1e-3


def _peak(wl, token):
    """Queries whose largest logit lies at a shared token."""
    q = wl.q_tokens(1)
    G = wl.Hq // wl.Hkv
    for b in range(wl.B):
        k = wl.kv(wl.B - 1)[0][token]  # [Hkv, D]
        q[b, 0] += np.repeat(k, G, 0).reshape(wl.Hq, wl.D)
    return W.bf16_round(q)


@pytest.mark.parametrize("size", [2.0 ** -8, 2.0 ** -12, 2.0 ** -20])
@pytest.mark.parametrize("out_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("zeros", [(0, 32), (0, 64), (352, 384), (640, 704)])
@pytest.mark.parametrize("peak", [None, 16, 365])
def test_runs_of_zero_v_beside_small_v(size, out_dtype, zeros, peak):
    """32 or 64 tokens with V = 0 (their scales are 0): in the first half tile, over the first tile, in the middle, at
    the end; with the rows' largest logit in the run or elsewhere."""
    wl = _scale_v(_one_group("tiny_int8", [690, 704, 704], 704, 91), lambda t: 0.0 if zeros[0] <= t < zeros[1] else size)
    c = _Call(wl, "int8", [0, 3], [704], splits=1, out_dtype=out_dtype, q=None if peak is None else _peak(wl, peak))
    c.launch(checked=True)
    _check(c, size)


def _shared_only(size_of, lens=(704, 700, 690), seed=92, name="tiny_int8"):
    """No own pages (the decode kernel's P x scale has a range of its own)."""
    return _scale_v(_one_group(name, list(lens), max(lens), seed), size_of)


@pytest.mark.parametrize("size", [2.0 ** -60, 2.0 ** -100, 2.0 ** -112, 2.0 ** -118, 2.0 ** 110])
@pytest.mark.parametrize("out_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", ["tiny_int8", "serving_int8"])
@pytest.mark.parametrize("splits", [1, 3])
def test_v_near_the_ends_of_its_range(size, out_dtype, name, splits):
    wl = _shared_only(lambda t: size, name=name)
    c = _Call(wl, "int8", [0, 3], [704], splits=splits, out_dtype=out_dtype)
    c.launch(checked=True)
    _check(c, size)


@pytest.mark.parametrize("out_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("first,later", [(2.0 ** -112, 1.0), (1.0, 2.0 ** -112), (2.0 ** -118, 2.0 ** 110), (0.0, 2.0 ** -118),
                                         (2.0 ** -118, 0.0)])
@pytest.mark.parametrize("at", [16, 352, 640])
def test_v_of_two_sizes(out_dtype, first, later, at):
    """The small part weighs as much as the large one in the sum of weights, whatever is left of it in the result."""
    wl = _shared_only(lambda t: first if t < at else later)
    c = _Call(wl, "int8", [0, 3], [704], splits=1, out_dtype=out_dtype)
    c.launch(checked=True)
    _check(c, max(first, later))


@pytest.mark.parametrize("fmt", ["int8", "nvfp4", "bf16"])
@pytest.mark.parametrize("out_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("splits", [1, 4])
def test_a_nan_logit_of_a_shared_token_is_not_lost(fmt, out_dtype, splits):
    """K of one token and head is NaN: the rows that see it are NaN (not the result without the prompt); a sequence
    that ends before it, another group and the other heads are as without it."""
    wl = _share(W.make("tiny_int8", lens=("list", [700, 710, 290, 400, 410]), seed=93), [0, 3, 5], [640, 384])
    gs = H.global_scales(wl, fmt)
    c = _Call(wl, fmt, [0, 3, 5], [640, 384], splits=splits, out_dtype=out_dtype, gs=gs)
    c.launch(checked=True)
    out, lse = c.out.clone(), c.lse.clone()
    kc, _, ks, _ = c.cache.views()
    page, head, row = int(wl.block_tables[0, 300 // 16]), 1, 300 % 16
    if fmt == "bf16":
        kc[page, head, row].view(torch.bfloat16)[7] = float("nan")
    elif fmt == "int8":
        ks[page, head, row] = float("nan")
    else:
        ks[page, head, row, 3] = 0x7F
    c.launch(checked=True)
    G = wl.Hq // wl.Hkv
    hit = torch.zeros((wl.B, 1, wl.Hq), dtype=torch.bool, device="cuda")
    hit[:2, :, G * head:G * head + G] = True
    assert torch.all(torch.isnan(c.out[hit])) and torch.all(torch.isnan(c.lse[hit]))
    assert torch.equal(c.out[~hit], out[~hit]) and torch.equal(c.lse[~hit], lse[~hit])


def test_a_nan_query_row():
    wl = _one_group("tiny_int8", [600, 610], 592, 94)
    q = wl.q_tokens(1)
    q[1, 0, 5, 17] = np.nan
    for fmt in ("int8", "bf16"):
        c = _Call(wl, fmt, [0, 2], [592], splits=3, q=q)
        c.launch(checked=True)
        bad = torch.zeros((2, 1, wl.Hq), dtype=torch.bool, device="cuda")
        bad[1, 0, 5] = True
        assert torch.all(torch.isnan(c.out[bad])) and torch.all(torch.isnan(c.lse[bad]))
        assert torch.all(torch.isfinite(c.out[~bad])) and torch.all(torch.isfinite(c.lse[~bad]))


@pytest.mark.parametrize("out_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("which", ["one", "some", "all"])
def test_scales_of_either_sign(out_dtype, which):
    """The append writes scales >= 0, but a pool may hold any: code x scale is the value, as in the decode."""
    wl = _one_group("tiny_int8", [704, 700, 690], 704, 96)
    c = _Call(wl, "int8", [0, 3], [704], splits=2, out_dtype=out_dtype)
    _, _, ks, vs = c.cache.views()
    pools = H.oracle_pools(wl, "int8")
    rng = np.random.default_rng(7)
    sign = {"one": np.ones(ks.shape, np.float32), "some": rng.choice(np.float32([-1, 1]), ks.shape),
            "all": np.full(ks.shape, -1, np.float32)}[which]
    if which == "one":
        sign[int(wl.block_tables[0, 9]), 2, 5] = -1
    for dev, name in ((ks, "k_scales"), (vs, "v_scales")):
        pools[name] *= sign
        dev.mul_(torch.from_numpy(sign).cuda())
    c.launch(checked=True)
    _check(c, 1.0, pools)


@pytest.mark.parametrize("fmt,value", [("int8", "nan"), ("int8", "inf"), ("nvfp4", "nan"), ("bf16", "nan"), ("bf16", "inf")])
@pytest.mark.parametrize("out_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,splits,name", [(1, 1, "tiny_int8"), (3, 1, "serving_int8"), (3, 4, "tiny_int8")])
def test_v_behind_a_rows_last_token_does_not_reach_it(T, splits, name, fmt, out_dtype, value):
    """V of shared token 304 holds a NaN or an infinity.  Sequences of 700 and 710 tokens see it, one of 305 with its
    last query token only, one of 290 and an empty one never: their rows are as without it, and of the rows that see it
    the columns that it is in are not finite.  (Two results of one row differ by their roundings: the tolerance is
    twice that of each.)"""
    wl = _share(W.make(name, lens=("list", [700, 710, 290, 305, 0]), seed=99), [0, 5], [640])
    gs = H.global_scales(wl, fmt)
    c = _Call(wl, fmt, [0, 5], [640], T=T, splits=splits, out_dtype=out_dtype, gs=gs)
    c.launch(checked=True)
    out, lse = c.out.clone(), c.lse.clone()
    _, vc, _, vs = c.cache.views()
    page, head, row = int(wl.block_tables[0, 304 // 16]), 1, 304 % 16
    cols = slice(0, wl.D)
    if fmt == "bf16":
        vc[page, head, row].view(torch.bfloat16)[7] = float(value)
        cols = slice(7, 8)
    elif fmt == "int8":
        vs[page, head, row] = float(value)
    else:
        vs[page, head, row, 3] = 0x7F
        cols = slice(48, 64)
    c.launch(checked=True)
    G = wl.Hq // wl.Hkv
    hit = torch.zeros(c.out.shape, dtype=torch.bool, device="cuda")
    heads = slice(G * head, G * head + G)
    hit[:2, :, heads, cols] = True
    hit[3, T - 1, heads, cols] = True
    assert not torch.any(torch.isfinite(c.out[hit]))
    # INT8: the weights are formed as 2^(z - m + d), d the exponent of a half tile's V under the largest of the range (here
    # that of the NaN or infinity: d = -60); a number below 2^7 is rounded by up to 2^-18, and so is the weight
    fin = torch.isfinite(lse)
    assert torch.equal(torch.isfinite(c.lse), fin) and (c.lse[fin] - lse[fin]).abs().max() <= 2.0 ** -17
    others = torch.ones(wl.Hq, dtype=torch.bool)
    others[heads] = False
    assert torch.equal(c.out[:, :, others], out[:, :, others]) and torch.equal(c.lse[:, :, others], lse[:, :, others])
    a, b = c.out[~hit].float(), out[~hit].float()
    assert torch.all((a - b).abs() <= (4e-3 if out_dtype == "f32" else torch.clamp(2.0 ** -7 * b.abs(), min=2e-2)))
