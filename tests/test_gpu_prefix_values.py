"""kvq_paged_prefix_attention where single values are unlike the rest: runs of V = 0, V near the ends of its range.

Tolerance: as in test_gpu_prefix_range.py, the decode tests' bounds scaled with the size of V."""
import numpy as np
import pytest

from quantized_paged_kv_gb300 import workloads as W
from tests import harness as H
from tests.test_gpu_prefix import _Call, _one_group
from tests.test_gpu_prefix_range import _check, _scale_v

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    H.ensure_built()


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
